"""The routed-expert layer around the deltas: tokens sorted by expert and back, and matrix products with bias, delta,
activation and residual in one pass, dense or over the experts' rows.

As in the rest of the binding, every function only marshals tensors into the C ABI of ``include/lora_delta.h`` (where
layouts, limits and errors are stated) on torch's current CUDA stream, and turns a nonzero status into ``LoraError``.
Tensors must be on the current device.
"""
from __future__ import annotations

import functools

import torch

from ._lib import lib
from .serve import _DTYPES, _check, _err_at, _Fixed, _fn, _raw_stream

_ACTIVATIONS = {"none": 0, None: 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def _here(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on {t.device}, not on the current device")


def _matrix(t, name, dtype, rows, width, here):
    """Pointer and row stride of a [rows, width] tensor with adjacent columns on device `here`; rows may lie apart."""
    if t.dtype is dtype and t.get_device() == here and t.shape == (rows, width):
        ld, step = t.stride()
        if step == 1 or width <= 1:
            return t.data_ptr(), ld
    _here(t, name)
    raise ValueError(f"{name} must be {dtype} [{rows}, {width}] with adjacent columns, got {t.dtype} {tuple(t.shape)}")


def _whole(t, name, dtype, shape, here):
    """Pointer of a contiguous tensor of this shape on device `here`, or None."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == here and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _here(t, name)
    raise ValueError(f"{name} must be a contiguous {dtype} tensor {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _rows_dtype(t, name):
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be bfloat16 or float16, not {t.dtype}")
    return t.dtype


class MoePlan(_Fixed):
    """What ``lora_moe_dispatch`` writes for ``T`` tokens of ``top_k`` experts among ``E``: ``seg_start`` [E + 1], ``pair_row``
    [T, top_k], ``row_pair``, ``row_expert`` and ``row_lora`` [T * top_k], all int32.  Until then no pair has a row."""

    def __init__(self, T: int, top_k: int, E: int, device="cuda"):
        if torch.device(device).type != "cuda":
            raise ValueError(f"a plan's tensors are the GPU's, not {device}'s")
        if T < 0 or top_k < 1 or E < 1:
            raise ValueError(f"a plan of {T} tokens, {top_k} experts each of {E}")
        self.T, self.top_k, self.E, self.n_rows = int(T), int(top_k), int(E), int(T) * int(top_k)

        def ints(*shape, value=-1):
            return torch.full(shape, value, dtype=torch.int32, device=device)

        self.seg_start, self.pair_row = ints(self.E + 1, value=0), ints(self.T, self.top_k)
        self.row_pair, self.row_expert, self.row_lora = (ints(self.n_rows) for _ in range(3))
        self._device = self.seg_start.get_device()
        self._seg, self._pair = self.seg_start.data_ptr(), self.pair_row.data_ptr()
        self._out = (self._seg, self.row_pair.data_ptr(), self._pair, self.row_expert.data_ptr(), self.row_lora.data_ptr())


def _plan_here(plan):
    """The current device, which the plan has to be on."""
    here = torch._C._cuda_getDevice()
    if plan._device != here:
        raise ValueError(f"the plan is on device {plan._device}, not on the current one")
    return here


def lora_moe_dispatch(rows, x, topk_ids, plan: MoePlan, lora_ids=None, expert_map=None, err=None, stream=None) -> MoePlan:
    """Sort the tokens by expert into ``plan`` and their rows ``x`` [T, H] into ``rows`` [T * top_k, H].

    ``topk_ids`` [T, top_k] int32, -1 for a padded token; ``lora_ids`` [T] int32 the tokens' adapters; ``expert_map`` int32 the
    global experts' numbers on this rank, -1 elsewhere.  The gradient for x is ``lora_moe_combine(grad_x, grad_rows, plan)``."""
    T, k = plan.T, plan.top_k
    H, dtype = x.shape[-1], _rows_dtype(x, "x")
    here = _plan_here(plan)
    x_at, ld_x = _matrix(x, "x", dtype, T, H, here)
    rows_at, ld_rows = _matrix(rows, "rows", dtype, plan.n_rows, H, here)
    n_map = 0
    if expert_map is not None:
        n_map = expert_map.numel()
        expert_map = _whole(expert_map, "expert_map", torch.int32, (n_map,), here)
    _check("lora_moe_dispatch", _fn.lora_moe_dispatch(
        rows_at, ld_rows, *plan._out, x_at, ld_x, _whole(topk_ids, "topk_ids", torch.int32, (T, k), here),
        _whole(lora_ids, "lora_ids", torch.int32, (T,), here), expert_map, n_map, T, k, plan.E, H, _err_at(err), _raw_stream(stream)))
    return plan


def lora_moe_combine(out, rows, plan: MoePlan, weights=None, residual=None, stream=None):
    """``out[t] = residual[t] + sum_j weights[t, j] rows[plan.pair_row[t, j]]``, over the pairs that have a row.

    ``weights`` [T, top_k] float32 (1 without); ``residual`` [T, H] may be ``out`` itself.  Without either it is the gradient
    of ``lora_moe_dispatch``."""
    T, H, dtype = plan.T, out.shape[-1], _rows_dtype(out, "out")
    here = _plan_here(plan)
    out_at, ld_out = _matrix(out, "out", dtype, T, H, here)
    rows_at, ld_rows = _matrix(rows, "rows", dtype, plan.n_rows, H, here)
    res_at, ld_res = (None, 0) if residual is None else _matrix(residual, "residual", dtype, T, H, here)
    _check("lora_moe_combine", _fn.lora_moe_combine(
        out_at, ld_out, rows_at, ld_rows, plan._pair, _whole(weights, "weights", torch.float32, (T, plan.top_k), here), res_at, ld_res,
        T, plan.top_k, H, _DTYPES[dtype], _raw_stream(stream)))


def lora_moe_combine_grad(grad_rows, grad_weights, grad_out, rows, plan: MoePlan, weights=None, stream=None):
    """The gradient of ``lora_moe_combine`` for its rows, into ``grad_rows`` (rows that no pair has stay as they were), and for
    its weights, into ``grad_weights`` [T, top_k] float32 or None.  That for the residual is ``grad_out`` itself."""
    T, H, dtype = plan.T, grad_out.shape[-1], _rows_dtype(grad_out, "grad_out")
    here = _plan_here(plan)
    go_at, ld_go = _matrix(grad_out, "grad_out", dtype, T, H, here)
    rows_at, ld_rows = _matrix(rows, "rows", dtype, plan.n_rows, H, here)
    gr_at, ld_gr = _matrix(grad_rows, "grad_rows", dtype, plan.n_rows, H, here)
    _check("lora_moe_combine_grad", _fn.lora_moe_combine_grad(
        gr_at, ld_gr, _whole(grad_weights, "grad_weights", torch.float32, (T, plan.top_k), here), go_at, ld_go, rows_at, ld_rows,
        plan._pair, _whole(weights, "weights", torch.float32, (T, plan.top_k), here), T, plan.top_k, H, _DTYPES[dtype],
        _raw_stream(stream)))


def _activation(name):
    if name not in _ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(k for k in _ACTIVATIONS if k)}, got {name!r}")
    return _ACTIVATIONS[name]


def _epilogue(delta, residual, dtype, n, N, width, here):
    d = (None, 0) if delta is None else _matrix(delta, "delta", dtype, n, N, here)
    r = (None, 0) if residual is None else _matrix(residual, "residual", dtype, n, width, here)
    return *d, *r


@functools.lru_cache(maxsize=4096)
def _linear_bytes(n, groups):
    return int(lib().lora_linear_workspace_size(n, groups))


def lora_linear_workspace(device="cuda") -> torch.Tensor:
    """A workspace for ``lora_linear`` and ``lora_moe_linear`` of any size, ready for its first use."""
    L = lib()
    ws = torch.empty(int(L.lora_linear_workspace_size(2 ** 31 - 1, 1)), dtype=torch.uint8, device=device)
    ws[:int(L.lora_linear_zeroed_bytes())].zero_()
    return ws


# One workspace per (device, stream) for callers that pass none, as for the attention: calls on one stream run in order
# and may share it.  A graph gets its own, since its replays may run beside calls on the stream of its capture.
_LINEAR_WS: dict = {}


def _linear_workspace(workspace, n, groups, device, stream, raw):
    """Pointer and bytes of the workspace of a call."""
    if workspace is not None:
        _here(workspace, "workspace")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    elif not _linear_bytes(n, groups):
        return None, 0
    elif stream is not None:
        with torch.cuda.stream(stream):
            return _linear_workspace(None, n, groups, device, None, raw)
    elif torch._C._cuda_isCurrentStreamCapturing():
        workspace = lora_linear_workspace(torch.device("cuda", device))  # zeroed by each replay
    else:
        workspace = _LINEAR_WS.get((device, raw))
        if workspace is None:
            workspace = _LINEAR_WS[(device, raw)] = lora_linear_workspace(torch.device("cuda", device))
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def lora_linear(out, x, weight, bias=None, delta=None, residual=None, activation="none", gated: bool = False,
                workspace=None, err=None, stream=None):
    """``out = act(x weight^T + bias + delta) + residual``; gated: ``act(z[:, :I]) * z[:, I:] + residual`` of z [n, 2 I].

    ``x`` [n, k_in], ``weight`` [n_out, k_in], ``bias`` [n_out], ``delta`` [n, n_out] (what the LoRA calls leave: it goes
    ahead of the activation), all bfloat16 or all float16, and ``residual`` as ``out``, which it may be itself.  ``activation``:
    "none", "relu", "silu", "gelu" (by erf) or "gelu_tanh".  No argument may lie in ``workspace`` or hold ``err``.  ``out`` may be
    an adapter's weights only where other work on the stream comes between this call and the delta that reads them."""
    here = torch._C._cuda_getDevice()
    dtype, n = _rows_dtype(x, "x"), x.shape[0]
    if weight.dim() != 2:
        raise ValueError(f"weight must be [n_out, k_in], got {tuple(weight.shape)}")
    N, K = weight.shape
    width = N // 2 if gated else N
    x_at, ld_x = _matrix(x, "x", dtype, n, K, here)
    w_at, ld_w = _matrix(weight, "weight", dtype, N, K, here)
    out_at, ld_out = _matrix(out, "out", dtype, n, width, here)
    raw = _raw_stream(stream)
    ws, ws_bytes = _linear_workspace(workspace, n, 1, here, stream, raw)
    _check("lora_linear", _fn.lora_linear(
        out_at, ld_out, x_at, ld_x, n, K, w_at, ld_w, N, _whole(bias, "bias", dtype, (N,), here),
        *_epilogue(delta, residual, dtype, n, N, width, here), _activation(activation), 1 if gated else 0, _DTYPES[dtype],
        ws, ws_bytes, _err_at(err), raw))


def lora_moe_linear(out, rows, weight, plan: MoePlan, bias=None, delta=None, residual=None, activation="none",
                    gated: bool = False, workspace=None, err=None, stream=None):
    """``lora_linear`` of the sorted ``rows`` [T * top_k, k_in] of ``plan``, expert e's with ``weight[e]`` of [E, n_out, k_in] and
    ``bias[e]`` of [E, n_out].  ``delta`` and ``residual`` are in the rows' order.  Rows behind the last expert's are left as
    they were."""
    dtype, n = _rows_dtype(rows, "rows"), plan.n_rows
    _here(weight, "weight")
    here = _plan_here(plan)
    if weight.dtype is not dtype or weight.dim() != 3 or weight.shape[0] != plan.E:
        raise ValueError(f"weight must be {dtype} [{plan.E}, n_out, k_in], got {weight.dtype} {tuple(weight.shape)}")
    E, N, K = weight.shape
    stride_w, ld_w, step = weight.stride()
    if step != 1 and K > 1:
        raise ValueError("weight's columns must be adjacent")
    width = N // 2 if gated else N
    x_at, ld_x = _matrix(rows, "rows", dtype, n, K, here)
    out_at, ld_out = _matrix(out, "out", dtype, n, width, here)
    raw = _raw_stream(stream)
    ws, ws_bytes = _linear_workspace(workspace, n, E, here, stream, raw)
    _check("lora_moe_linear", _fn.lora_moe_linear(
        out_at, ld_out, x_at, ld_x, n, K, plan._seg, E, weight.data_ptr(), ld_w if N > 1 else K, stride_w, N,
        _whole(bias, "bias", dtype, (E, N), here), *_epilogue(delta, residual, dtype, n, N, width, here), _activation(activation),
        1 if gated else 0, _DTYPES[dtype], ws, ws_bytes, _err_at(err), raw))
