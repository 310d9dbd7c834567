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
