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


_torch = _lib = _raw_stream = _current_device = None


def _load():
    """The library's handle; the first call also brings in torch."""
    global _torch, _lib, _raw_stream, _current_device
    import torch
    _torch = torch
    # the current stream's handle without building a Stream object (1 us less), where torch has it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _current_device = torch.cuda.current_device
    _lib = _base().load()
    return _lib


def _device(t) -> int:
    """The index of the CUDA device that a call's first tensor lives on."""
    try:
        index = t.get_device()
    except AttributeError:
        raise TypeError("tensors must be torch.Tensor") from None
    if index < 0:
        raise ValueError("tensors must live on a CUDA device")
    return index


def _ptr(name, t, dtype, shape, index, contiguous=True):
    """Checks a tensor (None passes; shape None = any) and returns its address."""
    if t is None:
        return None
    try:
        if (t.dtype is dtype and t.get_device() == index and (shape is None or t.shape == shape) and
                (not contiguous or t.is_contiguous())):
            return t.data_ptr()
    except AttributeError:
        raise TypeError(f"{name} must be a torch.Tensor") from None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the call's tensors are on cuda:{index}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    raise ValueError(f"{name} must be contiguous")


def _elsewhere(index, stream):
    """The context that a call has to enter first, so that the device is current and its current stream the
    one asked for (what is allocated then belongs to it); None where both already hold."""
    if stream is None:
        return None if _current_device() == index else _torch.cuda.device(index)
    return _torch.cuda.stream(stream if hasattr(stream, "cuda_stream") else _torch.cuda.ExternalStream(int(stream), device=index))


def _fail(rc):
    _base()._raise(rc)


def _rows(name, t, dims):
    """Checks the dimensions of a tensor whose last one must be contiguous; returns its strides."""
    st = t.stride()
    if len(st) != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    return st


def _scratch(workspace, nbytes, index, dev):
    """(tensor, address, bytes) of a call's workspace: the given one, or a new one of nbytes()."""
    if workspace is None:
        n = nbytes()
        if n == 0:
            _fail(_base().ERR_INVALID_ARG)
        workspace = _torch.empty(n, dtype=_torch.uint8, device=dev)
    return workspace, _ptr("workspace", workspace, _torch.uint8, None, index, dev), workspace.numel()


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
    lib = _lib or _load()
    first = q if q is not None else k
    if first is None:
        raise ValueError("pass q, k or both")
    index, dev, dtype, i32 = _device(first), first.device, first.dtype, _torch.int32
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return rotary(q, positions, inv_freq, k=k, v=v, q_out=q_out, k_out=k_out, v_out=v_out, slot=slot, amplitude=amplitude,
                          interleaved=interleaved, inverse=inverse, status=status)
    if dtype is _torch.bfloat16:
        code = OUT_BF16
    elif dtype is _torch.float32:
        code = OUT_F32
    else:
        raise TypeError(f"rotary takes bfloat16 or float32, got {dtype}")
    freq = inv_freq
    if type(freq) is not np.ndarray or freq.dtype != np.float64 or freq.ndim != 1 or not freq.flags.c_contiguous:
        freq = np.ascontiguousarray(freq, dtype=np.float64).reshape(-1)
    if (v is None) != (v_out is None):
        raise ValueError("pass v and v_out together")
    if v is not None and k is None:
        raise ValueError("v needs k")
    if slot is not None and (k is None or k_out is None):
        raise ValueError("slot needs k and k_out")
    _rows("q" if q is not None else "k", first, 3)
    n, _, dh = first.shape
    a, capacity = [], n
    if q is None:
        a += (None, 0, 0, None, 0, 0, 0)
    else:
        if q_out is None:
            q_out = _torch.empty(q.shape, dtype=dtype, device=dev)
        st, so = q.stride(), _rows("q_out", q_out, 3)
        a += (q.data_ptr(), st[0], st[1], _ptr("q_out", q_out, dtype, q.shape, index, False), so[0], so[1], q.shape[1])
    if k is None:
        a += (None, 0, 0, None, 0, 0, 0)
    else:
        st, ks = _rows("k", k, 3), k.shape
        hkv = ks[1]
        if ks[0] != n or ks[2] != dh:
            raise ValueError("k must be [n, Hkv, Dh] like q")
        if k_out is None:
            k_out = _torch.empty(ks, dtype=dtype, device=dev)
        ko = _store_rows("k_out", k_out, ks, slot is None)
        capacity, so = ko.shape[0], ko.stride()
        a += (_ptr("k", k, dtype, None, index, False), st[0], st[1], _ptr("k_out", ko, dtype, None, index, False), so[0], so[1],
              hkv)
    if v is None:
        a += (None, 0, 0, None, 0, 0)
    else:
        st = _rows("v", v, 3)
        vo = _store_rows("v_out", v_out, k.shape, slot is None)
        so = vo.stride()
        if vo.shape[0] != capacity:
            raise ValueError("v_out must have as many rows as k_out")
        a += (_ptr("v", v, dtype, k.shape, index, False), st[0], st[1], _ptr("v_out", vo, dtype, None, index, False), so[0], so[1])
    rc = lib.dflash_rotary(*a, _ptr("positions", positions, i32, (n,), index), _ptr("slot", slot, i32, (n,), index), n, capacity,
                           dh, 2 * freq.shape[0], freq.tobytes(), float(amplitude), 1 if interleaved else 0, 1 if inverse else 0, code,
                           _ptr("status", status, i32, (1,), index), _raw_stream(index))
    if rc:
        _fail(rc)
    return q_out, k_out


def _store_rows(name, t, like, dense):
    """A destination of k or v as [rows, Hkv, Dh]; dense: as many rows as k."""
    if t.dim() == 4:
        t = t.view(-1, t.shape[2], t.shape[3])
    _rows(name, t, 3)
    s = t.shape
    if s[1] != like[1] or s[2] != like[2] or (dense and s[0] != like[0]):
        raise ValueError(f"{name} must be [{'n' if dense else 'capacity'}, Hkv, Dh]")
    return t


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
    lib = _lib or _load()
    index, dev, bf16, i32 = _device(q), q.device, _torch.bfloat16, _torch.int32
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return decode_attention_paged(q, k_pool, v_pool, block_table, seq_lens, max_ctx_len=max_ctx_len, out=out, lse=lse,
                                          return_lse=return_lse, workspace=workspace, scale=scale, window=window,
                                          out_dtype=out_dtype, status=status)
    sq = _rows("q", q, 3)
    n, hq, dh = q.shape
    if k_pool.dim() != 4 or block_table.dim() != 2:
        raise ValueError("k_pool must be [num_pages, page_size, Hkv, Dh] and block_table [N, max_pages]")
    pages, page, hkv, kdh = k_pool.shape
    width, stb = block_table.shape[1], block_table.stride()
    if kdh != dh:
        raise ValueError(f"q has head_dim {dh}, the pools {kdh}")
    if hq > 1 and sq[1] != dh and n:
        raise ValueError("q: the heads of a sequence must be contiguous")
    if width > 1 and stb[1] != 1:
        raise ValueError("block_table: a row must be contiguous")
    max_ctx_len, window = int(max_ctx_len), int(window)
    if out_dtype != OUT_BF16 and out_dtype != OUT_F32:
        raise ValueError("out_dtype must be OUT_BF16 or OUT_F32")
    odt = _torch.float32 if out_dtype == OUT_F32 else bf16
    p_q, p_k = _ptr("q", q, bf16, None, index, False), _ptr("k_pool", k_pool, bf16, None, index)
    p_v, p_t = _ptr("v_pool", v_pool, bf16, k_pool.shape, index), _ptr("block_table", block_table, i32, (n, width), index, False)
    p_l = _ptr("seq_lens", seq_lens, i32, (n,), index)
    if out is None:
        out = _torch.empty((n, hq, dh), dtype=odt, device=dev)
    if lse is None and return_lse:
        lse = _torch.empty((n, hq), dtype=_torch.float32, device=dev)
    workspace, p_w, w_bytes = _scratch(
        workspace, lambda: lib.dflash_decode_workspace_size(n, hq, hkv, dh, max_ctx_len, window), index, dev)
    rc = lib.dflash_decode_attention_paged(
        p_q, sq[0] if n > 1 else hq * dh, p_k, p_v, p_t, stb[0] if n > 1 else width, p_l, n, hq, hkv, dh, pages, page, width,
        max_ctx_len, float(scale), window, out_dtype, _ptr("out", out, odt, (n, hq, dh), index),
        _ptr("lse", lse, _torch.float32, (n, hq), index), p_w, w_bytes, _ptr("status", status, i32, (1,), index), _raw_stream(index))
    if rc:
        _fail(rc)
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
    lib = _lib or _load()
    index, dev, f32, i32, flag = _device(logits), logits.device, _torch.float32, _torch.int32, _torch.bool
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return beam_select(logits, scores, beams_out=beams_out, finished=finished, eos=eos, out=out, workspace=workspace)
    st = _rows("logits", logits, 3)
    n, w, vocab = logits.shape
    k = w if beams_out is None else int(beams_out)
    dtype = logits.dtype
    if dtype is f32:
        code = OUT_F32
    elif dtype is _torch.bfloat16:
        code = OUT_BF16
    else:
        raise TypeError(f"logits must be bfloat16 or float32, got {dtype}")
    if k <= 0:
        raise ValueError("beams_out must be positive")
    shape = (n, k)
    p_s, p_f = _ptr("scores", scores, f32, (n, w), index), _ptr("finished", finished, flag, (n, w), index)
    out = dict(out) if out else {}
    ptr = []
    for name, dt in zip(BEAM_OUTPUTS, (f32, i32, i32, flag)):
        t = out.get(name)
        if t is None:
            t = out[name] = _torch.empty(shape, dtype=dt, device=dev)
            ptr.append(t.data_ptr())
        else:
            ptr.append(_ptr(name, t, dt, shape, index))
    workspace, p_w, w_bytes = _scratch(workspace, lambda: lib.dflash_beam_workspace_size(n, w, k, vocab, code), index, dev)
    rc = lib.dflash_beam_select(logits.data_ptr(), st[0], st[1], p_s, p_f, n, w, k, vocab, int(eos), code, *ptr, p_w, w_bytes, _raw_stream(index))
    if rc:
        _fail(rc)
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


def _table(block_table, page_refs, index):
    """(rows, width, stride, address of the table, of the counts, pages)."""
    st = block_table.stride()
    if len(st) != 2 or page_refs.dim() != 1:
        raise ValueError("block_table must be [N, max_pages] and page_refs [num_pages]")
    n, width = block_table.shape
    if width > 1 and st[1] != 1:
        raise ValueError("block_table: a row must be contiguous")
    if n > 1 and st[0] < width:
        raise ValueError("block_table: rows must not overlap")
    return (n, width, st[0] if n > 1 else width, _ptr("block_table", block_table, _torch.int32, None, index, False),
            _ptr("page_refs", page_refs, _torch.int32, None, index), page_refs.shape[0])


def _pools(pools, num_pages, index):
    """(host array of addresses, count, bytes per page, rows per page) of a list of pools."""
    size = page = None
    addr = []
    for i, t in enumerate(pools):
        s = t.shape
        if t.get_device() != index or not t.is_contiguous() or len(s) < 2 or s[0] != num_pages:
            raise ValueError(f"pool {i} must be a contiguous [num_pages, page_size, ...] tensor on cuda:{index}")
        b = t.element_size() * math.prod(s[1:])
        if size is not None and (b != size or s[1] != page):
            raise ValueError("all pools must have pages of the same size")
        size, page = b, s[1]
        addr.append(t.data_ptr())
    return (ctypes.c_void_p * max(1, len(addr)))(*addr), len(addr), size or 0, page


def fork_pages(parent, seq_lens, block_table, page_refs, *, status=None, stream=None) -> None:
    """Row i of block_table [N, max_pages] and seq_lens [N] becomes row parent[i]'s, in place; -1 frees it.

    page_refs [num_pages] int32 counts the table entries that name a page (0 = free) and follows. Nothing
    is copied: reserve_pages gives a row its own copy of a shared page before it is written.
    """
    lib = _lib or _load()
    index, dev, i32 = _device(block_table), block_table.device, _torch.int32
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return fork_pages(parent, seq_lens, block_table, page_refs, status=status)
    n, width, stride, p_t, p_r, pages = _table(block_table, page_refs, index)
    if parent.dim() > 1:
        parent = parent.view(-1)
    rc = lib.dflash_fork_pages(_ptr("parent", parent, i32, (n,), index), _ptr("seq_lens", seq_lens, i32, (n,), index), p_t, stride,
                               p_r, n, width, pages, _ptr("status", status, i32, (1,), index), _raw_stream(index))
    if rc:
        _fail(rc)


def reserve_pages(new_start_loc, seq_lens, block_table, page_refs, pools, *, num_new, page_size=None, advance=False,
                  slots=None, positions=None, workspace=None, status=None, stream=None):
    """Makes room for new_start_loc[r+1] - new_start_loc[r] rows behind every sequence's stored ones.

    Pages are taken lowest first, row by row; a page that other rows share is replaced by an own copy (of
    the sequence's rows, in every tensor of `pools` [num_pages, page_size, ...]) before it is written. Returns
    (slots, positions) int32 [num_new]: the pool row and the position of every new row; -1 and 0 where a
    sequence was refused (no pages left, or its table is full), which status reports. advance=True also
    adds the new rows to seq_lens. page_size is needed only with an empty list of pools.
    """
    lib = _lib or _load()
    index, dev, i32 = _device(block_table), block_table.device, _torch.int32
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return reserve_pages(new_start_loc, seq_lens, block_table, page_refs, pools, num_new=num_new, page_size=page_size,
                                 advance=advance, slots=slots, positions=positions, workspace=workspace, status=status)
    n, width, stride, p_t, p_r, pages = _table(block_table, page_refs, index)
    arr, count, page_bytes, page = _pools(pools, pages, index)
    if page is None:
        if page_size is None:
            raise ValueError("page_size is needed without pools")
        page = int(page_size)
    elif page_size is not None and page_size != page:
        raise ValueError("page_size is not the pools'")
    num_new = int(num_new)
    if num_new < 0:
        raise ValueError("num_new must be >= 0")
    if slots is None:
        slots = _torch.empty(num_new, dtype=i32, device=dev)
    if positions is None:
        positions = _torch.empty(num_new, dtype=i32, device=dev)
    workspace, p_w, w_bytes = _scratch(workspace, lambda: lib.dflash_pages_workspace_size(n, pages), index, dev)
    rc = lib.dflash_reserve_pages(
        _ptr("new_start_loc", new_start_loc, i32, (n + 1,), index), _ptr("seq_lens", seq_lens, i32, (n,), index), p_t, stride, p_r,
        arr, count, page_bytes, n, num_new, width, page, pages, 1 if advance else 0,
        _ptr("slots", slots, i32, (num_new,), index), _ptr("positions", positions, i32, (num_new,), index), p_w, w_bytes,
        _ptr("status", status, i32, (1,), index), _raw_stream(index))
    if rc:
        _fail(rc)
    return slots, positions


def compact_pages(block_table, page_refs, pools, *, used=None, workspace=None, status=None, stream=None):
    """Moves the used pages to the lowest ids, in every tensor of `pools`, with tables and counts.

    Returns `used`, an int32 device word: the number of pages in use, which are now the first ones.
    """
    lib = _lib or _load()
    index, dev, i32 = _device(block_table), block_table.device, _torch.int32
    away = _elsewhere(index, stream)
    if away is not None:
        with away:
            return compact_pages(block_table, page_refs, pools, used=used, workspace=workspace, status=status)
    n, width, stride, p_t, p_r, pages = _table(block_table, page_refs, index)
    arr, count, page_bytes, _ = _pools(pools, pages, index)
    if used is None:
        used = _torch.empty(1, dtype=i32, device=dev)
    workspace, p_w, w_bytes = _scratch(workspace, lambda: lib.dflash_pages_workspace_size(n, pages), index, dev)
    rc = lib.dflash_compact_pages(p_t, stride, p_r, arr, count, page_bytes, n, width, pages,
                                  _ptr("used", used, i32, (1,), index), p_w, w_bytes, _ptr("status", status, i32, (1,), index),
                                  _raw_stream(index))
    if rc:
        _fail(rc)
    return used
