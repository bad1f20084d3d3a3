"""Decoding over the paged store: bindings of the calls that a decode step makes.

    rotary(...)                 -> dflash_rotary
    decode_attention_paged(...) -> dflash_decode_attention_paged
    beam_select(...)            -> dflash_beam_select
    fork_pages(...)             -> dflash_fork_pages
    reserve_pages(...)          -> dflash_reserve_pages
    compact_pages(...)          -> dflash_compact_pages

Like the rest of the package these only marshal arguments. All tensors of a call live on one device;
the call runs there, on `stream` (default: that device's current stream). Outputs and workspaces that
a call allocates belong to that stream.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import numpy as np

OUT_BF16, OUT_F32 = 0, 1


def declare(lib) -> None:
    """Argument types of the library's decode entry points."""
    P, I32, I64, F32, F64, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                                 ctypes.c_size_t)
    sig = {
        "dflash_rotary": (I32, [P, I64, I64, P, I64, I64, I32, P, I64, I64, P, I64, I64, I32, P, I64, I64, P, I64, I64, P,
                                P, I64, I64, I32, I32, P, F64, I32, I32, I32, P, P]),
        "dflash_decode_workspace_size": (SZ, [I32, I32, I32, I32, I32, I32]),
        "dflash_decode_attention_paged": (I32, [P, I64, P, P, P, I64, P, I32, I32, I32, I32, I64, I32, I32, I32, F32, I32,
                                                I32, P, P, P, SZ, P, P]),
        "dflash_beam_workspace_size": (SZ, [I32, I32, I32, I32, I32]),
        "dflash_beam_select": (I32, [P, I64, I64, P, P, I32, I32, I32, I32, I32, I32, P, P, P, P, P, SZ, P]),
        "dflash_pages_workspace_size": (SZ, [I32, I64]),
        "dflash_fork_pages": (I32, [P, P, P, I64, P, I32, I32, I64, P, P]),
        "dflash_reserve_pages": (I32, [P, P, P, I64, P, P, I32, I64, I32, I64, I32, I32, I64, I32, P, P, P, SZ, P, P]),
        "dflash_compact_pages": (I32, [P, I64, P, P, I32, I64, I32, I32, I64, P, P, SZ, P, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args


def _base():
    import speculative_decoding_draft_rmsnorm_gb300 as pkg
    return pkg


_NO_GUARD = contextlib.nullcontext()


class _Call:
    """The device and stream of a call; allocations made inside belong to that stream."""

    __slots__ = ("lib", "device", "handle", "guard")

    def __init__(self, first, stream):
        import torch
        if not isinstance(first, torch.Tensor) or not first.is_cuda:
            raise ValueError("tensors must live on a CUDA device")
        self.lib = _base().load()
        self.device = first.device
        index = self.device.index
        if stream is None:
            s = torch.cuda.current_stream(index)
            self.handle = s.cuda_stream
            self.guard = _NO_GUARD if torch.cuda.current_device() == index else torch.cuda.device(index)
        else:
            s = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), device=self.device)
            self.handle = s.cuda_stream
            self.guard = torch.cuda.stream(s)

    def tensor(self, name, t, dtype, shape, contiguous=True):
        """Checks a tensor (None passes) and returns its address."""
        if t is None:
            return None
        import torch
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the call's tensors are on {self.device}")
        if t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if shape is not None and t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def run(self, fn, *args):
        rc = fn(*args, self.handle)
        if rc != 0:
            _base()._raise(rc)


def _rows(name, t, dims):
    """Checks the dimensions of a tensor whose last one must be contiguous."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")


def _workspace(call, workspace, nbytes):
    import torch
    if nbytes == 0:
        _base()._raise(_base().ERR_INVALID_ARG)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=call.device)
    return call.tensor("workspace", workspace, torch.uint8, None), workspace.numel()


# ------------------------------------------------------------------------------------- rotary
def rotary_frequencies(rotary_dim: int, theta: float = 1e6, *, scaling: str = "none", factor: float = 1.0,
                       original_len: int = 0, fast: float = 32.0, slow: float = 1.0):
    """(angle per position of every pair, float64 numpy [rotary_dim / 2]; amplitude) for `rotary`.

    scaling: "none": theta^(-2i/d); "linear": those divided by `factor` (positions interpolated);
    "base": theta stretched to theta * factor^(d / (d - 2)), so that the lowest frequency is divided by
    `factor` and the highest kept; "parts": pairs that turn more than `fast` times over `original_len`
    positions are kept, those below `slow` turns are divided by `factor`, with a ramp over the pair
    index between, and the amplitude is 0.1 ln(factor) + 1.
    """
    d = int(rotary_dim)
    if d < 2 or d % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not (theta > 1.0 and math.isfinite(theta)) or not (factor >= 1.0 and math.isfinite(factor)):
        raise ValueError("theta must be above 1 and factor at least 1")
    i = np.arange(d // 2, dtype=np.float64)
    if scaling == "base":
        base = theta * factor ** (d / (d - 2.0)) if d > 2 else theta
        return base ** (-2.0 * i / d), 1.0
    freq = theta ** (-2.0 * i / d)
    if scaling == "none":
        return freq, 1.0
    if scaling == "linear":
        return freq / factor, 1.0
    if scaling != "parts":
        raise ValueError(f"unknown scaling {scaling!r}")
    if original_len <= 0 or not fast > slow > 0:
        raise ValueError("parts needs original_len > 0 and fast > slow > 0")

    def pair_of(turns):  # the pair index that turns so often over original_len positions
        return d * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(theta))

    lo, hi = max(0, math.floor(pair_of(fast))), min(d - 1, math.ceil(pair_of(slow)))
    ramp = np.clip((i - lo) / max(hi - lo, 1e-3), 0.0, 1.0)
    return freq * (1 - ramp) + freq / factor * ramp, 0.1 * math.log(factor) + 1.0


def rotary(q, positions, inv_freq, *, k=None, v=None, q_out=None, k_out=None, v_out=None, slot=None, amplitude=1.0,
           interleaved=False, inverse=False, status=None, stream=None):
    """Rotary positions of q [n, Hq, Dh] (and k [n, Hkv, Dh]); returns (q_out, k_out).

    q, k, v: bf16 or f32 with any strides but a contiguous last dimension; positions [n] int32;
    inv_freq: host float64 [rotary_dim / 2] (see rotary_frequencies); the head's elements behind
    rotary_dim are copied. Outputs default to new contiguous tensors; q_out = q and k_out = k work in
    place. With slot [n] int32, k (and v) go to rows slot[t] of k_out (and v_out) [capacity, Hkv, Dh] or
    [num_pages, page_size, Hkv, Dh]; -1 = not stored. inverse=True applies the transpose: the gradient
    of the inputs from that of the outputs. q may be None.
    """
    import torch
    first = q if q is not None else k
    if first is None:
        raise ValueError("pass q, k or both")
    c = _Call(first, stream)
    dtype = first.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"rotary takes bfloat16 or float32, got {dtype}")
    freq = inv_freq if isinstance(inv_freq, np.ndarray) else np.asarray(inv_freq, dtype=np.float64)
    if freq.dtype != np.float64 or freq.ndim != 1 or not freq.flags.c_contiguous:
        freq = np.ascontiguousarray(freq, dtype=np.float64).reshape(-1)
    _rows("q" if q is not None else "k", first, 3)
    n, _, dh = first.shape
    if (v is None) != (v_out is None):
        raise ValueError("pass v and v_out together")
    if v is not None and k is None:
        raise ValueError("v needs k")
    if slot is not None and (k is None or k_out is None):
        raise ValueError("slot needs k and k_out")
    p_pos = c.tensor("positions", positions, torch.int32, (n,))
    p_slot = c.tensor("slot", slot, torch.int32, (n,))
    p_status = c.tensor("status", status, torch.int32, (1,))
    with c.guard:
        parts = [None, 0, 0, None, 0, 0, 0, None, 0, 0, None, 0, 0, 0, None, 0, 0, None, 0, 0]
        capacity = n
        if q is not None:
            if q_out is None:
                q_out = torch.empty(q.shape, dtype=dtype, device=c.device)
            _rows("q_out", q_out, 3)
            parts[0:7] = [c.tensor("q", q, dtype, None, False), q.stride(0), q.stride(1),
                          c.tensor("q_out", q_out, dtype, q.shape, False), q_out.stride(0), q_out.stride(1), q.shape[1]]
        if k is not None:
            _rows("k", k, 3)
            if k.shape[0] != n or k.shape[2] != dh:
                raise ValueError("k must be [n, Hkv, Dh] like q")
            hkv = k.shape[1]
            if k_out is None:
                k_out = torch.empty(k.shape, dtype=dtype, device=c.device)

            def store(name, t):
                if t.dim() == 4:
                    t = t.view(-1, t.shape[2], t.shape[3])
                _rows(name, t, 3)
                if t.shape[1] != hkv or t.shape[2] != dh or (slot is None and t.shape[0] != n):
                    raise ValueError(f"{name} must be [{'capacity' if slot is not None else 'n'}, Hkv, Dh]")
                return t

            ko = store("k_out", k_out)
            capacity = ko.shape[0]
            parts[7:14] = [c.tensor("k", k, dtype, None, False), k.stride(0), k.stride(1),
                           c.tensor("k_out", ko, dtype, None, False), ko.stride(0), ko.stride(1), hkv]
            if v is not None:
                _rows("v", v, 3)
                vo = store("v_out", v_out)
                if vo.shape[0] != capacity:
                    raise ValueError("v_out must have as many rows as k_out")
                parts[14:20] = [c.tensor("v", v, dtype, k.shape, False), v.stride(0), v.stride(1),
                                c.tensor("v_out", vo, dtype, None, False), vo.stride(0), vo.stride(1)]
        c.run(c.lib.dflash_rotary, *parts, p_pos, p_slot, n, capacity, dh, 2 * freq.shape[0], freq.ctypes.data,
              float(amplitude), int(bool(interleaved)), int(bool(inverse)), OUT_F32 if dtype == torch.float32 else OUT_BF16,
              p_status)
    return q_out, k_out


# ------------------------------------------------------------------------------------- attention
def decode_workspace_size(num_reqs, hq, hkv, dh, max_ctx_len, window=0) -> int:
    n = _base().load().dflash_decode_workspace_size(num_reqs, hq, hkv, dh, int(max_ctx_len), int(window))
    if n == 0:
        _base()._raise(_base().ERR_INVALID_ARG)
    return int(n)


def decode_attention_paged(q, k_pool, v_pool, block_table, seq_lens, *, max_ctx_len, out=None, lse=None, return_lse=False,
                           workspace=None, scale=0.0, window=0, out_dtype=OUT_BF16, status=None, stream=None):
    """Attention of one new token per sequence, q [N, Hq, Dh], over its stored rows (its own among them).

    k_pool / v_pool [num_pages, page_size, Hkv, Dh] bf16; block_table [N, max_pages] int32 (its rows may
    be strided); seq_lens [N] int32 on the device; window > 0: the last `window` rows only. Returns out
    [N, Hq, Dh], or (out, lse [N, Hq] f32) with return_lse=True or an lse tensor. A length of 0 gives
    zeros and -inf. max_ctx_len bounds the lengths (grid and workspace size only).
    """
    import torch
    c = _Call(q, stream)
    _rows("q", q, 3)
    n, hq, dh = q.shape
    if k_pool.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, Dh] and block_table [N, max_pages]")
    pages, page, hkv, kdh = k_pool.shape
    width = block_table.shape[1]
    bf16, i32 = torch.bfloat16, torch.int32
    if kdh != dh:
        raise ValueError(f"q has head_dim {dh}, the pools {kdh}")
    if hq > 1 and n and q.stride(1) != dh:
        raise ValueError("q: the heads of a sequence must be contiguous")
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: a row must be contiguous")
    p_q = c.tensor("q", q, bf16, None, False)
    p_k = c.tensor("k_pool", k_pool, bf16, None)
    p_v = c.tensor("v_pool", v_pool, bf16, k_pool.shape)
    p_t = c.tensor("block_table", block_table, i32, (n, width), False)
    p_l = c.tensor("seq_lens", seq_lens, i32, (n,))
    p_status = c.tensor("status", status, i32, (1,))
    odt = torch.float32 if out_dtype == OUT_F32 else bf16
    lib = c.lib
    with c.guard:
        if out is None:
            out = torch.empty((n, hq, dh), dtype=odt, device=c.device)
        if lse is None and return_lse:
            lse = torch.empty((n, hq), dtype=torch.float32, device=c.device)
        p_o = c.tensor("out", out, odt, (n, hq, dh))
        p_lse = c.tensor("lse", lse, torch.float32, (n, hq))
        if workspace is None:
            p_w, w_bytes = _workspace(c, None, lib.dflash_decode_workspace_size(n, hq, hkv, dh, max_ctx_len, window))
        else:
            p_w, w_bytes = _workspace(c, workspace, 1)
        c.run(lib.dflash_decode_attention_paged, p_q, q.stride(0) if n > 1 else hq * dh, p_k, p_v, p_t,
              block_table.stride(0) if n > 1 else width, p_l, n, hq, hkv, dh, pages, page, width, max_ctx_len, scale, window,
              out_dtype, p_o, p_lse, p_w, w_bytes, p_status)
    return out if lse is None else (out, lse)


# ------------------------------------------------------------------------------------- beams
BEAM_OUTPUTS = ("scores", "tokens", "parents", "finished")


def beam_select(logits, scores, *, beams_out=None, finished=None, eos=-1, out=None, workspace=None, stream=None) -> dict:
    """The best continuations of every request's beams, as a dict named as BEAM_OUTPUTS.

    logits [N, W, vocab] bf16 or f32 (last dimension contiguous), scores [N, W] f32 (-inf: not live),
    finished [N, W] bool; K = beams_out (default W) of W * vocab candidates are kept, best first, ties to
    the lowest index. Outputs [N, K]: scores f32, tokens int32, parents int32 (row r * W + w, as
    fork_pages takes them), finished bool; slots without a candidate hold -inf, -1, -1, False.
    `out` may hold preallocated outputs, e.g. for graph capture.
    """
    import torch
    c = _Call(logits, stream)
    _rows("logits", logits, 3)
    n, w, vocab = logits.shape
    k = w if beams_out is None else int(beams_out)
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    dt = OUT_F32 if logits.dtype == torch.float32 else OUT_BF16
    p_x = c.tensor("logits", logits, logits.dtype, None, False)
    p_s = c.tensor("scores", scores, torch.float32, (n, w))
    p_f = c.tensor("finished", finished, torch.bool, (n, w))
    if k <= 0:
        raise ValueError("beams_out must be positive")
    lib = c.lib
    with c.guard:
        out = dict(out) if out else {}
        ptr = []
        for name, dtype in zip(BEAM_OUTPUTS, (torch.float32, torch.int32, torch.int32, torch.bool)):
            if name not in out:
                out[name] = torch.empty((n, k), dtype=dtype, device=c.device)
            ptr.append(c.tensor(name, out[name], dtype, (n, k)))
        if workspace is None:
            p_w, w_bytes = _workspace(c, None, lib.dflash_beam_workspace_size(n, w, k, vocab, dt))
        else:
            p_w, w_bytes = _workspace(c, workspace, 1)
        c.run(lib.dflash_beam_select, p_x, logits.stride(0), logits.stride(1), p_s, p_f, n, w, k, vocab, int(eos), dt, *ptr,
              p_w, w_bytes)
    return out


def beam_workspace_size(num_reqs, beams, beams_out, vocab, dtype=OUT_BF16) -> int:
    n = _base().load().dflash_beam_workspace_size(num_reqs, beams, beams_out, vocab, dtype)
    if n == 0:
        _base()._raise(_base().ERR_INVALID_ARG)
    return int(n)


# ------------------------------------------------------------------------------------- pages
def pages_workspace_size(num_reqs, num_pages) -> int:
    n = _base().load().dflash_pages_workspace_size(num_reqs, num_pages)
    if n == 0:
        _base()._raise(_base().ERR_INVALID_ARG)
    return int(n)


def _table(c, block_table, page_refs, rows=None):
    import torch
    if block_table.dim() != 2 or page_refs.dim() != 1:
        raise ValueError("block_table must be [N, max_pages] and page_refs [num_pages]")
    n, width = block_table.shape
    if width > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: a row must be contiguous")
    if n > 1 and block_table.stride(0) < width:
        raise ValueError("block_table: rows must not overlap")
    p_t = c.tensor("block_table", block_table, torch.int32, None, False)
    p_r = c.tensor("page_refs", page_refs, torch.int32, None)
    return n, width, block_table.stride(0) if n > 1 else width, p_t, p_r, page_refs.shape[0]


def _pools(c, pools, num_pages):
    """(host array of addresses, count, bytes per page, rows per page) of a list of pools."""
    size = page = None
    for i, t in enumerate(pools):
        if t.device != c.device or not t.is_contiguous() or t.dim() < 2 or t.shape[0] != num_pages:
            raise ValueError(f"pool {i} must be a contiguous [num_pages, page_size, ...] tensor on {c.device}")
        b = t.element_size() * math.prod(t.shape[1:])
        if size is not None and (b != size or t.shape[1] != page):
            raise ValueError("all pools must have pages of the same size")
        size, page = b, t.shape[1]
    arr = (ctypes.c_void_p * max(1, len(pools)))(*[t.data_ptr() for t in pools])
    return arr, len(pools), size or 0, page


def fork_pages(parent, seq_lens, block_table, page_refs, *, status=None, stream=None) -> None:
    """Row i of block_table [N, max_pages] and seq_lens [N] becomes row parent[i]'s, in place; -1 frees it.

    page_refs [num_pages] int32 counts the table entries that name a page (0 = free) and follows. Nothing
    is copied: reserve_pages gives a row its own copy of a shared page before it is written.
    """
    import torch
    c = _Call(block_table, stream)
    n, width, stride, p_t, p_r, pages = _table(c, block_table, page_refs)
    p_p = c.tensor("parent", parent.view(-1) if isinstance(parent, torch.Tensor) and parent.dim() > 1 else parent, torch.int32, (n,))
    p_l = c.tensor("seq_lens", seq_lens, torch.int32, (n,))
    p_status = c.tensor("status", status, torch.int32, (1,))
    with c.guard:
        c.run(c.lib.dflash_fork_pages, p_p, p_l, p_t, stride, p_r, n, width, pages, p_status)


def reserve_pages(new_start_loc, seq_lens, block_table, page_refs, pools, *, num_new, page_size=None, advance=False,
                  slots=None, positions=None, workspace=None, status=None, stream=None):
    """Makes room for new_start_loc[r+1] - new_start_loc[r] rows behind every sequence's stored ones.

    Pages are taken lowest first, row by row; a page that other rows share is replaced by an own copy (of
    the sequence's rows, in every tensor of `pools` [num_pages, page_size, ...]) before it is written. Returns
    (slots, positions) int32 [num_new]: the pool row and the position of every new row; -1 and 0 where a
    sequence was refused (no pages left, or its table is full), which status reports. advance=True also
    adds the new rows to seq_lens. page_size is needed only with an empty list of pools.
    """
    import torch
    c = _Call(block_table, stream)
    n, width, stride, p_t, p_r, pages = _table(c, block_table, page_refs)
    arr, count, page_bytes, page = _pools(c, pools, pages)
    if page is None:
        if page_size is None:
            raise ValueError("page_size is needed without pools")
        page = int(page_size)
    elif page_size is not None and page_size != page:
        raise ValueError("page_size is not the pools'")
    num_new = int(num_new)
    if num_new < 0:
        raise ValueError("num_new must be >= 0")
    i32 = torch.int32
    p_s = c.tensor("new_start_loc", new_start_loc, i32, (n + 1,))
    p_l = c.tensor("seq_lens", seq_lens, i32, (n,))
    p_status = c.tensor("status", status, i32, (1,))
    with c.guard:
        if slots is None:
            slots = torch.empty(num_new, dtype=i32, device=c.device)
        if positions is None:
            positions = torch.empty(num_new, dtype=i32, device=c.device)
        p_slots = c.tensor("slots", slots, i32, (num_new,))
        p_pos = c.tensor("positions", positions, i32, (num_new,))
        if workspace is None:
            p_w, w_bytes = _workspace(c, None, c.lib.dflash_pages_workspace_size(n, pages))
        else:
            p_w, w_bytes = _workspace(c, workspace, 1)
        c.run(c.lib.dflash_reserve_pages, p_s, p_l, p_t, stride, p_r, arr, count, page_bytes, n, num_new, width, page, pages,
              int(bool(advance)), p_slots, p_pos, p_w, w_bytes, p_status)
    return slots, positions


def compact_pages(block_table, page_refs, pools, *, used=None, workspace=None, status=None, stream=None):
    """Moves the used pages to the lowest ids, in every tensor of `pools`, with tables and counts.

    Returns `used`, an int32 device word: the number of pages in use, which are now the first ones.
    """
    import torch
    c = _Call(block_table, stream)
    n, width, stride, p_t, p_r, pages = _table(c, block_table, page_refs)
    arr, count, page_bytes, _ = _pools(c, pools, pages)
    p_status = c.tensor("status", status, torch.int32, (1,))
    with c.guard:
        if used is None:
            used = torch.empty(1, dtype=torch.int32, device=c.device)
        p_u = c.tensor("used", used, torch.int32, (1,))
        if workspace is None:
            p_w, w_bytes = _workspace(c, None, c.lib.dflash_pages_workspace_size(n, pages))
        else:
            p_w, w_bytes = _workspace(c, workspace, 1)
        c.run(c.lib.dflash_compact_pages, p_t, stride, p_r, arr, count, page_bytes, n, width, pages, p_u, p_w, w_bytes,
              p_status)
    return used
