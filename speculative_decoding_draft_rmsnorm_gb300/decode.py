"""Decoding over the paged store: bindings of the calls that a decode step makes.

    rotary(...)                 -> dflash_rotary
    decode_attention_paged(...) -> dflash_decode_attention_paged
    beam_select(...)            -> dflash_beam_select
    fork_pages(...)             -> dflash_fork_pages
    reserve_pages(...)          -> dflash_reserve_pages
    compact_pages(...)          -> dflash_compact_pages
and a step of sequences that share a prompt:
    rms_norm(...)                -> dflash_rms_norm
    rotary_axes(...)             -> dflash_rotary_axes
    shared_prefixes(...)         -> dflash_shared_prefixes
    decode_attention_shared(...) -> dflash_decode_attention_shared

Like the rest of the package these only marshal arguments (csrc/bind.cpp checks them and makes the call).
All tensors of a call live on one device; the call runs there, on `stream` (default: that device's current
stream). Outputs and workspaces that a call allocates belong to that stream. No call records a gradient; rotary,
whose inverse is one, and rms_norm refuse tensors that require it while gradients are recorded. Tensors that a call writes count
as changed in place.
"""
from __future__ import annotations

import ctypes
import math

import numpy as np

OUT_BF16, OUT_F32, OUT_E4M3 = 0, 1, 2


def declare(lib) -> None:
    """Argument types of the library's decode entry points."""
    P, I32, I64, F32, F64, SZ = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                                 ctypes.c_size_t)
    sig = {
        "dflash_rotary": (I32, [P, I64, I64, P, I64, I64, I32, P, I64, I64, P, I64, I64, I32, P, I64, I64, P, I64, I64, P,
                                P, I64, I64, I32, I32, P, F64, I32, I32, I32, P, P]),
        "dflash_rotary_axes": (I32, [P, I64, I64, P, I64, I64, I32, P, I64, I64, P, I64, I64, I32, P, I64, I64, P, I64, I64, P,
                                     I64, I32, P, P, I64, I64, I32, I32, P, F64, I32, I32, I32, P, P]),
        "dflash_rms_norm": (I32, [P, I64, P, I64, P, P, I64, P, I64, P, I64, I32, I32, I32, I32, I32, F32, P, P]),
        "dflash_shared_prefixes": (I32, [P, I64, P, P, I32, I32, I32, I32, P, P, P]),
        "dflash_decode_workspace_size": (SZ, [I32, I32, I32, I32, I32, I32]),
        "dflash_decode_attention_paged": (I32, [P, I64, P, P, P, I64, P, I32, I32, I32, I32, I64, I32, I32, I32, F32, I32,
                                                I32, P, P, P, SZ, P, P]),
        "dflash_shared_workspace_size": (SZ, [I32] * 7),
        "dflash_decode_attention_shared": (I32, [P, I64, P, P, P, I64, P, P, P, I32, I32, I32, I32, I32, I64, I32, I32, I32, F32,
                                                 I32, I32, P, P, P, SZ, I32, P, P]),
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


_bind = None  # the marshalling module (csrc/bind.cpp)


def _load():
    """Loads the marshalling module, and with it the library and torch, which it is built against."""
    global _bind
    import importlib.machinery
    import importlib.util

    import torch  # noqa: F401  (the module links to it)

    from . import _build
    _base().load()
    with _base()._lock:
        if _bind is None:
            path = _build.bind_path()
            if not _build.up_to_date(path):
                _build.build()
            loader = importlib.machinery.ExtensionFileLoader("_decode_bind", path)
            module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_decode_bind", loader))
            loader.exec_module(module)
            _bind = module
    return _bind


def _fail(rc):
    _base()._raise(rc)


def _on(stream, first):
    """The context in which `stream` (a torch stream or a raw handle) is current on the tensors' device."""
    import torch
    if not isinstance(first, torch.Tensor) or not first.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=first.device)
    elif stream.device != first.device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {first.device}")
    return torch.cuda.stream(stream)


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
    of the inputs from that of the outputs (none is recorded, so tensors that require one are refused
    outside torch.no_grad()). q may be None.
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, k if q is None else q):
            return rotary(q, positions, inv_freq, k=k, v=v, q_out=q_out, k_out=k_out, v_out=v_out, slot=slot, amplitude=amplitude,
                          interleaved=interleaved, inverse=inverse, status=status)
    if type(inv_freq) is not np.ndarray or inv_freq.dtype != np.float64 or not inv_freq.flags.c_contiguous:
        inv_freq = np.ascontiguousarray(inv_freq, dtype=np.float64)
    out = bind.rotary(q, positions, inv_freq, k, v, q_out, k_out, v_out, slot, amplitude, interleaved, inverse, status)
    if type(out) is int:
        _fail(out)
    return out


def rotary_sections(sections, *, interleaved=False):
    """The axis of every pair (uint8 numpy) for `rotary_axes`, from the number of pairs that each axis has.

    sections (16, 24, 24): pairs 0-15 follow axis 0, 16-39 axis 1, 40-63 axis 2. interleaved=True deals the
    axes out in turn, 0, 1, 2, 0, 1, 2, .., until each has its number.
    """
    left = [int(n) for n in sections]
    if not left or min(left) < 0 or len(left) > 255:
        raise ValueError("sections must be the axes' numbers of pairs")
    if not interleaved:
        return np.repeat(np.arange(len(left), dtype=np.uint8), left)
    turn = np.concatenate([np.arange(n) for n in left])  # of an axis: its 1st, 2nd, .. pair
    axis = np.repeat(np.arange(len(left), dtype=np.uint8), left)
    return axis[np.lexsort((axis, turn))]


def rotary_axes(q, positions, axes, inv_freq, *, k=None, v=None, q_out=None, k_out=None, v_out=None, slot=None, amplitude=1.0,
                interleaved=False, inverse=False, status=None, stream=None):
    """`rotary` with a position on each of several axes (time, height, width); returns (q_out, k_out).

    positions [A, n] int32, A <= 4 (an axis's positions contiguous, each axis with its own: no expanded row); axes: the axis of every pair, host integers
    [rotary_dim / 2] (see rotary_sections). Pair i of token t turns by positions[axes[i], t] * inv_freq[i].
    Everything else as in rotary; inverse=True is the gradient here too.
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, k if q is None else q):
            return rotary_axes(q, positions, axes, inv_freq, k=k, v=v, q_out=q_out, k_out=k_out, v_out=v_out, slot=slot,
                               amplitude=amplitude, interleaved=interleaved, inverse=inverse, status=status)
    if type(inv_freq) is not np.ndarray or inv_freq.dtype != np.float64 or not inv_freq.flags.c_contiguous:
        inv_freq = np.ascontiguousarray(inv_freq, dtype=np.float64)
    if type(axes) is not np.ndarray or not axes.flags.c_contiguous:
        axes = np.ascontiguousarray(axes)
    out = bind.rotary_axes(q, positions, inv_freq, k, v, q_out, k_out, v_out, slot, amplitude, interleaved, inverse, status, axes)
    if type(out) is int:
        _fail(out)
    return out


# ------------------------------------------------------------------------------------- norm
def rms_norm(x, weight, *, residual=None, out_dtype=None, group_size=0, eps=1e-6, out=None, residual_out=None, scales=None,
             status=None, stream=None):
    """RMS norm of x [n, d] (bf16 or f32), or of x + residual; returns (out, residual_out, scales).

    h = x + residual, rounded to their type, is residual_out (None without a residual) and what is normed:
    y = h * weight / sqrt(mean(h^2) + eps). weight [d]: bf16 or f32. out: y in x's type, or with
    out_dtype=OUT_E4M3 y / scale in 8 bits (torch.float8_e4m3fn) with scales f32 [n, 1], max |y| / 448 of every row,
    or [n, ceil(d / group_size)], of every group_size columns (a multiple of 16); scales is None otherwise.
    Rows may be strided; residual_out=residual, or =x, works in place, and so does out=x.
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, x):
            return rms_norm(x, weight, residual=residual, out_dtype=out_dtype, group_size=group_size, eps=eps, out=out,
                            residual_out=residual_out, scales=scales, status=status)
    got = bind.rms_norm(x, weight, residual, out_dtype, group_size, eps, out, residual_out, scales, status)
    if type(got) is int:
        _fail(got)
    return got


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
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, q):
            return decode_attention_paged(q, k_pool, v_pool, block_table, seq_lens, max_ctx_len=max_ctx_len, out=out, lse=lse,
                                          return_lse=return_lse, workspace=workspace, scale=scale, window=window,
                                          out_dtype=out_dtype, status=status)
    got = bind.decode_attention_paged(q, k_pool, v_pool, block_table, seq_lens, int(max_ctx_len), out, lse, return_lse, workspace,
                                      scale, int(window), out_dtype, status)
    if type(got) is int:
        _fail(got)
    return got


def shared_prefixes(block_table, seq_lens, group_start_loc, *, page_size, out=None, status=None, stream=None):
    """How many leading rows the sequences of every group hold in the same pages: int32 [groups].

    Group g is the rows group_start_loc[g] .. group_start_loc[g + 1] (int32 [groups + 1] on the device) of block_table
    [N, max_pages] and seq_lens [N]; sequences of length 0 are left out. What fork_pages shares, reserve_pages ends
    at the page that a sequence writes: call this behind it, once a step for all layers.
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, block_table):
            return shared_prefixes(block_table, seq_lens, group_start_loc, page_size=page_size, out=out, status=status)
    got = bind.shared_prefixes(block_table, seq_lens, group_start_loc, page_size, out, status)
    if type(got) is int:
        _fail(got)
    return got


def shared_workspace_size(num_reqs, num_groups, hq, hkv, dh, max_ctx_len, window=0) -> int:
    n = _base().load().dflash_shared_workspace_size(num_reqs, num_groups, hq, hkv, dh, int(max_ctx_len), int(window))
    if n == 0:
        _base()._raise(_base().ERR_INVALID_ARG)
    return int(n)


def decode_attention_shared(q, k_pool, v_pool, block_table, seq_lens, group_start_loc, prefix_lens, *, max_ctx_len, out=None,
                            lse=None, return_lse=False, workspace=None, scale=0.0, window=0, out_dtype=OUT_BF16, flags=0,
                            status=None, stream=None):
    """`decode_attention_paged` where the rows that a group of sequences shares are read once for all of them.

    Group g is the sequences group_start_loc[g] .. group_start_loc[g + 1] (int32 [groups + 1]); the first prefix_lens[g]
    rows (int32 [groups], see shared_prefixes) of its sequences that are so long lie in the same pages. Everything
    else, and the result, as in decode_attention_paged; the workspace is shared_workspace_size's. Calls with few rows let
    every sequence read its own, unless flags=FLAG_FORCE_SHARE.
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, q):
            return decode_attention_shared(q, k_pool, v_pool, block_table, seq_lens, group_start_loc, prefix_lens,
                                           max_ctx_len=max_ctx_len, out=out, lse=lse, return_lse=return_lse, workspace=workspace,
                                           scale=scale, window=window, out_dtype=out_dtype, flags=flags, status=status)
    got = bind.decode_attention_shared(q, k_pool, v_pool, block_table, seq_lens, int(max_ctx_len), out, lse, return_lse, workspace,
                                       scale, int(window), out_dtype, status, group_start_loc, prefix_lens, flags)
    if type(got) is int:
        _fail(got)
    return got


# ------------------------------------------------------------------------------------- beams
BEAM_OUTPUTS = ("scores", "tokens", "parents", "finished")


def beam_select(logits, scores, *, beams_out=None, finished=None, eos=-1, out=None, workspace=None, stream=None) -> dict:
    """The best continuations of every request's beams, as a dict named as BEAM_OUTPUTS.

    logits [N, W, vocab] bf16 or f32 (last dimension contiguous), scores [N, W] f32 (-inf: not live),
    finished [N, W] bool; K = beams_out (default W) of W * vocab candidates are kept, best first, ties to
    the lowest index. Outputs [N, K]: scores f32, tokens int32, parents int32 (row r * W + w, as
    fork_pages takes them), finished bool; slots without a candidate hold -inf, -1, -1, False.
    `out` may hold preallocated outputs, e.g. for graph capture. Outputs that the call makes lie in one allocation:
    each keeps all of it alive, and torch.save of one saves the storage of all (clone one to keep it alone).
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, logits):
            return beam_select(logits, scores, beams_out=beams_out, finished=finished, eos=eos, out=out, workspace=workspace)
    s, t, p, f = (out.get("scores"), out.get("tokens"), out.get("parents"), out.get("finished")) if out else (None,) * 4
    got = bind.beam_select(logits, scores, None if beams_out is None else int(beams_out), finished, int(eos), s, t, p, f, workspace)
    if type(got) is int:
        _fail(got)
    return dict(zip(BEAM_OUTPUTS, got))


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


def fork_pages(parent, seq_lens, block_table, page_refs, *, status=None, stream=None) -> None:
    """Row i of block_table [N, max_pages] and seq_lens [N] becomes row parent[i]'s, in place; -1 frees it.

    page_refs [num_pages] int32 counts the table entries that name a page (0 = free) and follows. Nothing
    is copied: reserve_pages gives a row its own copy of a shared page before it is written.
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, block_table):
            return fork_pages(parent, seq_lens, block_table, page_refs, status=status)
    got = bind.fork_pages(parent, seq_lens, block_table, page_refs, status)
    if type(got) is int:
        _fail(got)


def reserve_pages(new_start_loc, seq_lens, block_table, page_refs, pools, *, num_new, page_size=None, advance=False,
                  slots=None, positions=None, workspace=None, status=None, stream=None):
    """Makes room for new_start_loc[r+1] - new_start_loc[r] rows behind every sequence's stored ones.

    Pages are taken lowest first, row by row; a page that other rows share is replaced by an own copy (of
    the sequence's rows, in every tensor of `pools` [num_pages, page_size, ...]) before it is written. Returns
    (slots, positions) int32 [num_new]: the pool row and the position of every new row; -1 and 0 where a
    sequence was refused (no pages left, or its table is full), which status reports. advance=True also
    adds the new rows to seq_lens. page_size is needed only with an empty list of pools.
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, block_table):
            return reserve_pages(new_start_loc, seq_lens, block_table, page_refs, pools, num_new=num_new, page_size=page_size,
                                 advance=advance, slots=slots, positions=positions, workspace=workspace, status=status)
    got = bind.reserve_pages(new_start_loc, seq_lens, block_table, page_refs, pools, num_new, page_size, advance, slots,
                            positions, workspace, status)
    if type(got) is int:
        _fail(got)
    return got


def compact_pages(block_table, page_refs, pools, *, used=None, workspace=None, status=None, stream=None):
    """Moves the used pages to the lowest ids, in every tensor of `pools`, with tables and counts.

    Returns `used`, an int32 device word: the number of pages in use, which are now the first ones.
    """
    bind = _bind or _load()
    if stream is not None:
        with _on(stream, block_table):
            return compact_pages(block_table, page_refs, pools, used=used, workspace=workspace, status=status)
    got = bind.compact_pages(block_table, page_refs, pools, used, workspace, status)
    if type(got) is int:
        _fail(got)
    return got
