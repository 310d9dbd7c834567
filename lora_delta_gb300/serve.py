"""The serving step around the delta: the batch plan, the 4-bit key/value cache and attention
over it.

As in the rest of the binding, every function only marshals tensors into the C ABI of
``include/lora_delta.h`` (where layouts, limits and errors are stated) on torch's current CUDA
stream, and turns a nonzero status into ``LoraError``.
"""
from __future__ import annotations

import torch

from . import LoraError, _dev
from ._lib import lib

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def _check(name, rc):
    if rc:
        raise LoraError(name, rc)


class _Functions:
    """The library's functions, looked up once (``lib()`` loads it on the first call)."""

    def __getattr__(self, name):
        fn = getattr(lib(), name)
        setattr(self, name, fn)
        return fn


_fn = _Functions()


def _at(t):
    return None if t is None else t.data_ptr()


def _err_at(t):
    if t is None:
        return None
    if not t.is_cuda or t.dtype not in (torch.int32, torch.uint32) or t.numel() < 1:
        raise ValueError("err must be an int32 CUDA tensor, as new_error_word() makes it")
    return t.data_ptr()


def _raw_stream(stream):
    # (torch.cuda.current_stream() builds a Stream object, a third of a small call's time)
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _i32(t, name, size=0):
    if not t.is_cuda or t.dtype is not torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    if t.numel() < size:
        raise ValueError(f"{name} must have {size} entries, got {t.numel()}")
    return t.data_ptr()


def _table(t, n_reqs):
    """Pointer, row stride and pages a request of a block table."""
    if t.is_cuda and t.dtype is torch.int32 and t.dim() == 2:
        rows, pages = t.shape
        ld, step = t.stride()
        if rows >= n_reqs and (step == 1 or pages <= 1 or n_reqs == 0):
            return t.data_ptr(), ld, pages
    raise ValueError("block_table must be an int32 CUDA tensor [n_reqs, max_pages] with adjacent entries")


def _rows(t, name, heads, head_dim, dtype):
    """Pointer and row stride of a [n, heads, head_dim] tensor whose rows may lie apart."""
    if not t.is_cuda or t.dtype is not dtype:
        raise ValueError(f"{name} must be a {dtype} CUDA tensor")
    if t.dim() != 3 or t.shape[1:] != (heads, head_dim):
        raise ValueError(f"{name} must be [n, {heads}, {head_dim}], got {tuple(t.shape)}")
    ld, head, step = t.stride()
    if step != 1 or (head != head_dim and heads > 1):
        raise ValueError(f"{name}'s heads must lie next to one another")
    return t.data_ptr(), ld if t.shape[0] > 1 else heads * head_dim


class _Fixed:
    """An object whose attributes are set once: it keeps their tensors' addresses."""

    def __setattr__(self, name, value):
        if name in self.__dict__:
            raise AttributeError(f"{type(self).__name__}.{name} is fixed: write into it, or make another")
        super().__setattr__(name, value)


class BatchPlan(_Fixed):
    """What ``lora_batch_plan`` writes for a batch of up to ``n_reqs`` requests padded to ``n_rows``
    rows: ``row_start`` [n_reqs + 1], ``seq_len`` [n_reqs], ``row_req``, ``position``, ``seq_slot``
    [n_rows] int32 and ``slot_map`` [n_rows] int64."""

    def __init__(self, n_reqs: int, n_rows: int, page_size: int, device="cuda"):
        def ints(n):
            return torch.empty(n, dtype=torch.int32, device=device)

        if torch.device(device).type != "cuda":
            raise ValueError(f"a plan's tensors are the GPU's, not {device}'s")
        self.n_reqs, self.n_rows, self.page_size = int(n_reqs), int(n_rows), int(page_size)
        self.row_start, self.seq_len = ints(n_reqs + 1), ints(n_reqs)
        self.row_req, self.position, self.seq_slot = ints(n_rows), ints(n_rows), ints(n_rows)
        self.slot_map = torch.empty(n_rows, dtype=torch.int64, device=device)
        self._out = [t.data_ptr() for t in (self.row_start, self.seq_len, self.row_req,
                                            self.position, self.slot_map, self.seq_slot)]


def lora_batch_plan(plan: BatchPlan, ctx_len, new_len, block_table, req_slot=None, free_pages=None,
                    free_count=None, free_left=None, err=None, stream=None) -> BatchPlan:
    """The step's maps and new pages from the requests' lengths, into ``plan``'s tensors.

    ``ctx_len`` may be ``plan.seq_len``, the lengths that the plan's last step left.  ``free_pages`` /
    ``free_count`` [1] are the stack of free pages (a count past its entries is cut and reported in
    ``err``); the height that is left goes to ``free_left`` [1], or back into ``free_count`` where none
    is given."""
    B = plan.n_reqs
    table, ld, pages = _table(block_table, B)
    free = count = left = None
    cap = 0
    if free_pages is not None:
        cap = free_pages.numel()
        free, count = _i32(free_pages, "free_pages"), _i32(free_count, "free_count", 1)
        left = count if free_left is None else _i32(free_left, "free_left", 1)
    _check("lora_batch_plan", _fn.lora_batch_plan_bounded(
        _i32(ctx_len, "ctx_len", B), _i32(new_len, "new_len", B),
        None if req_slot is None else _i32(req_slot, "req_slot", B), B, plan.n_rows, plan.page_size,
        table, ld, pages, free, cap, count, left, *plan._out, _err_at(err), _raw_stream(stream)))
    return plan


def lora_pages_release(done, seq_len, block_table, page_size: int, free_pages, free_count, err=None,
                       stream=None):
    """The pages of the requests with ``done[b] != 0`` back onto the stack of free pages."""
    B = done.numel()
    table, ld, pages = _table(block_table, B)
    _check("lora_pages_release", _fn.lora_pages_release(
        _i32(done, "done"), _i32(seq_len, "seq_len", B), B, int(page_size), table, ld, pages,
        _i32(free_pages, "free_pages"), free_pages.numel(), _i32(free_count, "free_count", 1), _err_at(err),
        _raw_stream(stream)))


def lora_kv4_page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().lora_kv4_page_bytes(int(page_size), int(kv_heads), int(head_dim)))


class Kv4Cache(_Fixed):
    """A key/value cache held in 4 bits.

    ``pages`` is its memory, uint8 [num_pages, kv_heads, page_size / 16, tile bytes]; ``dtype``
    (bfloat16 or float16) is the type of the keys, values and queries beside it."""

    def __init__(self, pages: torch.Tensor, page_size: int, head_dim: int, dtype=torch.bfloat16):
        _dev(pages, "pages", torch.uint8)
        if dtype not in _DTYPES:
            raise ValueError(f"the cache's rows are bfloat16 or float16, not {dtype}")
        self.pages, self.page_size, self.head_dim, self.dtype = pages, int(page_size), int(head_dim), dtype
        self.num_pages, self.kv_heads = int(pages.shape[0]), int(pages.shape[1])
        want = lora_kv4_page_bytes(page_size, self.kv_heads, head_dim)
        if not want:
            raise ValueError(f"pages of {page_size} tokens and heads of {head_dim} are not supported")
        if pages.numel() != self.num_pages * want:
            raise ValueError(f"a page of this cache has {want} bytes")
        self._args = (pages.data_ptr(), self.num_pages, self.page_size, self.kv_heads, self.head_dim,
                      _DTYPES[dtype])

    @classmethod
    def empty(cls, num_pages: int, page_size: int, kv_heads: int, head_dim: int,
              dtype=torch.bfloat16, device="cuda") -> "Kv4Cache":
        """A cache of its own memory, its contents unspecified."""
        nbytes = lora_kv4_page_bytes(page_size, kv_heads, head_dim)
        if not nbytes:
            raise ValueError(f"pages of {page_size} tokens, {kv_heads} heads of {head_dim} are not supported")
        tiles = kv_heads * (page_size // 16)
        return cls(torch.empty(num_pages, kv_heads, page_size // 16, nbytes // tiles,
                               dtype=torch.uint8, device=device), page_size, head_dim, dtype)


def _store_or_read(name, cache, k, v, slot_map, err, stream):
    n, H, D = k.shape[0], cache.kv_heads, cache.head_dim
    if v.shape[0] != n:
        raise ValueError("k and v must have the same number of rows")
    if not slot_map.is_cuda or slot_map.dtype is not torch.int64 or not slot_map.is_contiguous():
        raise ValueError("slot_map must be a contiguous int64 CUDA tensor")
    if slot_map.numel() != n:
        raise ValueError(f"slot_map must have {n} entries, got {slot_map.numel()}")
    k_at, ld_k = _rows(k, "k", H, D, cache.dtype)
    v_at, ld_v = _rows(v, "v", H, D, cache.dtype)
    _check(name, getattr(_fn, name)(*cache._args, k_at, ld_k, v_at, ld_v, slot_map.data_ptr(), n, _err_at(err),
                                    _raw_stream(stream)))


def lora_kv4_append(cache: Kv4Cache, k, v, slot_map, err=None, stream=None):
    """Quantise the rows ``k``, ``v`` [n, kv_heads, head_dim] and store row i at ``slot_map[i]``
    (a negative slot is not stored).  The rows may be slices of a fused projection's output."""
    _store_or_read("lora_kv4_append", cache, k, v, slot_map, err, stream)


def lora_kv4_read(cache: Kv4Cache, k, v, slot_map, err=None, stream=None):
    """The values that stored rows stand for, into ``k``, ``v`` [n, kv_heads, head_dim]."""
    _store_or_read("lora_kv4_read", cache, k, v, slot_map, err, stream)


def lora_kv4_attention_workspace(device="cuda") -> torch.Tensor:
    """A workspace for ``lora_kv4_attention``, ready for its first use."""
    L = lib()
    ws = torch.empty(int(L.lora_kv4_attention_workspace_size()), dtype=torch.uint8, device=device)
    ws[:int(L.lora_kv4_attention_zeroed_bytes())].zero_()
    return ws


# One workspace per (device, stream) for callers that pass none: calls on one
# stream run in order and may share it.  A graph gets its own, since its replays
# may run on any stream, beside calls on the one that it was captured on.
_ATTN_WS: dict = {}


def _attn_workspace(device, stream, raw):
    if stream is not None:
        with torch.cuda.stream(stream):
            return _attn_workspace(device, None, raw)
    if torch._C._cuda_isCurrentStreamCapturing():
        return lora_kv4_attention_workspace(device)  # zeroed by each replay
    ws = _ATTN_WS.get((device.index, raw))
    if ws is None:
        ws = _ATTN_WS[(device.index, raw)] = lora_kv4_attention_workspace(device)
    return ws


def lora_kv4_attention(out, q, cache: Kv4Cache, block_table, row_start, seq_len, max_q_len: int,
                       scale: float | None = None, window: int = 0, lse=None, workspace=None,
                       err=None, stream=None):
    """Causal attention of the rows ``q`` [n, q_heads, head_dim] over the cache, into ``out``.

    ``row_start`` [n_reqs + 1] and ``seq_len`` [n_reqs] as ``lora_batch_plan`` writes them; a request's
    keys must be stored before.  ``max_q_len``: the most rows of one request.  ``scale`` defaults to
    head_dim ** -0.5; ``window`` > 0 limits a row to the last ``window`` tokens up to its own.  ``lse``
    [n, q_heads] float32 receives the log of the softmax's denominator."""
    n, q_heads, D = q.shape
    B = seq_len.numel()
    if out.shape[0] != n:
        raise ValueError("out and q must have the same number of rows")
    if lse is not None:
        _dev(lse, "lse", torch.float32)
        if lse.numel() != n * q_heads:
            raise ValueError("lse must be [n, q_heads]")
    raw = _raw_stream(stream)
    if workspace is None:
        workspace = _attn_workspace(q.device, stream, raw)
    else:
        _dev(workspace, "workspace")
    out_at, ld_out = _rows(out, "out", q_heads, cache.head_dim, cache.dtype)
    q_at, ld_q = _rows(q, "q", q_heads, cache.head_dim, cache.dtype)
    table, ld, pages = _table(block_table, B)
    _check("lora_kv4_attention", _fn.lora_kv4_attention(
        out_at, ld_out, q_at, ld_q, n, q_heads, *cache._args, table, ld, pages,
        _i32(row_start, "row_start", B + 1), _i32(seq_len, "seq_len"), B, max_q_len,
        D ** -0.5 if scale is None else scale, window, _at(lse), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _err_at(err), raw))
