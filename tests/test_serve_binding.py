"""What the binding of the serving-step operators keeps between calls, and what it refuses."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests.test_serve import attention_case, dev, host, ld, run_attention  # noqa: F401

gpu = pytest.mark.gpu


@gpu
def test_graphs_do_not_share_a_workspace_with_calls_or_one_another(ld, monkeypatch):  # noqa: F811
    """A call, then two captures on the same stream: three workspaces; replayed beside one another and
    beside calls, the results stay."""
    from lora_delta_gb300 import serve
    c = attention_case(np.random.default_rng(3), [(3000, 1), (10, 1), (700, 1)], 128, 2, 4, 16, torch.bfloat16)
    want = run_attention(ld, c)[0]
    used, call = [], serve._fn.lora_kv4_attention

    def record(*args):
        used.append(args[-4])  # (workspace, its bytes, error word, stream)
        return call(*args)

    monkeypatch.setattr(serve._fn, "lora_kv4_attention", record)
    cache = ld.Kv4Cache(dev(c["pages"], np.uint8), 16, 128)
    args = dev(c["table"]), dev(c["start"]), dev(c["seq"]), c["max_q"]
    outs, graphs, s = [torch.empty_like(c["q"]) for _ in range(4)], [], torch.cuda.Stream()
    torch.cuda.synchronize()
    ld.lora_kv4_attention(outs[0], c["q"], cache, *args, stream=s)
    torch.cuda.synchronize()
    for i in (1, 2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            ld.lora_kv4_attention(outs[i], c["q"], cache, *args)
    with torch.cuda.graph(torch.cuda.CUDAGraph()):  # by the argument, from another current stream's capture
        ld.lora_kv4_attention(outs[3], c["q"], cache, *args, stream=torch.cuda.current_stream())
    ld.lora_kv4_attention(outs[0], c["q"], cache, *args, stream=s)
    assert used[0] == used[4] and len(set(used[:3])) == 3 and used[3] != used[0]
    other = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(20):
        for g, t in zip(graphs, other):
            with torch.cuda.stream(t):
                g.replay()
        ld.lora_kv4_attention(outs[0], c["q"], cache, *args, stream=s)
    torch.cuda.synchronize()
    for out in outs[:3]:
        assert torch.equal(out, want)


@gpu
@pytest.mark.parametrize("B,top,in_place", [(700, 9, False), (700, 9, True), (4096, 3, False), (40, 2, True), (600, 1, False)])
def test_plan_steps_on_its_own_lengths(ld, B, top, in_place):  # noqa: F811
    """The lengths that a step leaves are the next one's: the same tensor in and out, with one CTA's rows and more."""
    from tests import serve_ref as ref
    rng, P, max_pages = np.random.default_rng(B + top), 16, 6
    ctx, slots = rng.integers(0, 40, B), rng.integers(-1, 9, B)
    table = np.full((B, max_pages), -1)
    order = rng.permutation(B * max_pages)
    held = -(-ctx // P)
    at = np.concatenate([[0], np.cumsum(held)])
    for b in range(B):
        table[b, :held[b]] = order[at[b]:at[b + 1]]
    free, count = order[at[-1]:], len(order) - at[-1]
    n = B * top + 3
    p, d_table, d_free, d_count = ld.BatchPlan(B, n, P), dev(table), dev(free), dev([count])
    left = None if in_place else dev([0])
    p.seq_len.copy_(dev(ctx))
    for _ in range(3):
        new, err = rng.integers(0, top + 1, B), ld.new_error_word()
        want = ref.plan(ctx, new, slots, n, P, table, max_pages, free, count)
        ld.lora_batch_plan(p, p.seq_len, dev(new), d_table, req_slot=dev(slots), free_pages=d_free, free_count=d_count,
                           free_left=left, err=err)
        assert ld.lora_get_error(err) == want["err"] == 0
        for name in ("row_start", "seq_len", "row_req", "position", "seq_slot", "slot_map"):
            assert np.array_equal(host(getattr(p, name)), want[name]), name
        assert np.array_equal(host(d_table), want["table"])
        ctx, table, count = want["seq_len"], want["table"], want["left"]
        if not in_place:
            d_count.copy_(left)
        assert int(d_count[0]) == count


def test_plan_refuses_outputs_that_share_memory_with_inputs():
    import ctypes

    import lora_delta_gb300 as ld
    from lora_delta_gb300.build import build
    build()
    at = [0x100000 * (i + 1) for i in range(16)]  # never dereferenced: the checks come first
    names = ["ctx", "new", "slot", "table", "free", "count", "left", "start", "seq", "req", "pos", "map", "aslot"]

    def plan(**kw):
        p = {**dict(zip(names, at)), **kw}
        v = {k: ctypes.c_void_p(x) for k, x in p.items()}
        return ld.lib().lora_batch_plan(v["ctx"], v["new"], v["slot"], 8, 40, 16, v["table"], 4, 4, v["free"], v["count"],
                                        v["left"], v["start"], v["seq"], v["req"], v["pos"], v["map"], v["aslot"], None, None)

    by = dict(zip(names, at))
    for name in ("new", "slot", "count"):
        for out in ("start", "seq", "req", "pos", "map", "aslot"):
            assert plan(**{out: by[name]}) == 1, (name, out)
    for out in ("start", "req", "pos", "map", "aslot", "left"):
        assert plan(**{out: by["ctx"]}) == 1, out
    assert plan(seq=by["ctx"] + 4) == 1 and plan(seq=by["ctx"] - 28) == 1
    assert plan(map=by["new"] - 8 * 40 + 16) == 1


@gpu
def test_attention_refuses_workspaces_that_it_cannot_use(ld):  # noqa: F811
    c = attention_case(np.random.default_rng(1), [(20, 1)], 64, 1, 2, 16, torch.bfloat16)
    want = run_attention(ld, c)[0]
    nbytes = int(ld.lib().lora_kv4_attention_workspace_size())
    for ws in (torch.zeros(nbytes, dtype=torch.uint8), torch.zeros(nbytes, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError):
            run_attention(ld, c, workspace=ws)
    with pytest.raises(ld.LoraError) as e:
        run_attention(ld, c, workspace=torch.zeros(nbytes // 4 - 1, dtype=torch.int32, device="cuda"))
    assert e.value.code == 5
    # bytes count, not entries
    assert torch.equal(run_attention(ld, c, workspace=torch.zeros(nbytes // 4 + 1, dtype=torch.int32, device="cuda"))[0], want)


@gpu
def test_error_words_are_checked(ld):  # noqa: F811
    c = attention_case(np.random.default_rng(1), [(20, 1)], 64, 1, 2, 16, torch.bfloat16)
    cache = ld.Kv4Cache(dev(c["pages"], np.uint8), 16, 64)
    k, slots, one = torch.zeros(1, 1, 64, device="cuda").bfloat16(), torch.zeros(1, dtype=torch.int64, device="cuda"), dev([1])
    p, table = ld.BatchPlan(1, 1, 16), dev(c["table"])
    args = c["q"], c["q"], cache, table, dev(c["start"]), dev(c["seq"]), 1
    for err in (torch.zeros(1, dtype=torch.int32), torch.zeros(1, device="cuda"), torch.zeros(0, dtype=torch.int32, device="cuda")):
        for call in (lambda: ld.lora_batch_plan(p, one, one, table, err=err), lambda: ld.lora_kv4_append(cache, k, k, slots, err=err),
                     lambda: ld.lora_kv4_read(cache, k, k, slots, err=err), lambda: ld.lora_kv4_attention(*args, err=err),
                     lambda: ld.lora_pages_release(one, one, table, 16, one, one, err=err)):
            with pytest.raises(ValueError):
                call()


@gpu
def test_plans_and_caches_keep_the_tensors_that_they_were_made_with(ld):  # noqa: F811
    """Their addresses are taken once, so a tensor put in another's place would not be written."""
    p, cache = ld.BatchPlan(2, 4, 16), ld.Kv4Cache.empty(2, 16, 1, 64)
    for obj, names in ((p, ("row_start", "seq_len", "row_req", "position", "slot_map", "seq_slot", "n_rows", "page_size")),
                       (cache, ("pages", "page_size", "head_dim", "dtype", "num_pages", "kv_heads"))):
        for name in names:
            with pytest.raises(AttributeError):
                setattr(obj, name, getattr(obj, name))


@gpu
@pytest.mark.parametrize("count", [6, 1000, 2 ** 31 - 1, -1, -2 ** 31])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan_does_not_take_pages_past_the_stack(ld, count, in_place):  # noqa: F811
    """A height above the stack's entries counts as full, one below 0 as empty; both are reported."""
    from tests import serve_ref as ref
    ctx, new, P, free = np.array([3, 0]), np.array([30, 9]), 16, np.array([11, 12, 13, 14, 15])
    table = np.full((2, 4), -1)
    table[0, 0] = 2
    want = ref.plan(ctx, new, None, 40, P, table, 4, free, min(max(count, 0), 5))
    p, err, left = ld.BatchPlan(2, 40, P), ld.new_error_word(), dev([77])
    d_table, d_count = dev(table), dev([count])
    ld.lora_batch_plan(p, dev(ctx), dev(new), d_table, free_pages=dev(free), free_count=d_count,
                       free_left=None if in_place else left, err=err)
    assert ld.lora_get_error(err) == ref.ERR_PAGE
    for name in ("row_start", "seq_len", "row_req", "position", "slot_map"):
        assert np.array_equal(host(getattr(p, name)), want[name]), name
    assert np.array_equal(host(d_table), want["table"])
    assert int((d_count if in_place else left)[0]) == want["left"]


def test_plans_are_made_on_the_gpu():
    """The kernel writes to their addresses, which must not be the host's."""
    import lora_delta_gb300 as ld
    for device in ("cpu", torch.device("cpu")):
        with pytest.raises(ValueError):
            ld.BatchPlan(2, 4, 16, device=device)
