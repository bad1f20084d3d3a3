"""The decode-step entry points: host arguments that are refused before a device is touched, and the
host-side frequency tables (CPU)."""
import ctypes
import math

import numpy as np
import pytest

import speculative_decoding_draft_rmsnorm_gb300 as D

F = ctypes.c_void_p(256)  # never dereferenced: validation fails first


def test_exports():
    lib = D.load()
    for n in ("dflash_rotary", "dflash_decode_attention_paged", "dflash_decode_workspace_size", "dflash_beam_select",
              "dflash_beam_workspace_size", "dflash_fork_pages", "dflash_reserve_pages", "dflash_compact_pages",
              "dflash_pages_workspace_size"):
        assert getattr(lib, n).argtypes


def _rotary(n=4, hq=2, hkv=1, dh=64, rd=64, freq=None, amp=1.0, inter=0, inverse=0, dtype=0, capacity=4, q=F, qo=F, k=F, ko=F, v=None,
            vo=None, slot=None, qs=(128, 64), qos=(128, 64)):
    f = np.full(max(1, rd // 2), 0.5) if freq is None else freq
    return D.load().dflash_rotary(q, *qs, qo, *qos, hq, k, 64, 64, ko, 64, 64, hkv, v, 64, 64, vo, 64, 64, F, slot, n, capacity, dh,
                                  rd, f.ctypes.data, amp, inter, inverse, dtype, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(rd=63), D.ERR_INVALID_ARG), (dict(rd=66), D.ERR_INVALID_ARG), (dict(rd=0), D.ERR_INVALID_ARG),
    (dict(dh=512, rd=512), D.ERR_UNSUPPORTED), (dict(dh=2048), D.ERR_UNSUPPORTED), (dict(dtype=2), D.ERR_INVALID_ARG),
    (dict(hq=0, hkv=0), D.ERR_INVALID_ARG), (dict(hq=-1), D.ERR_INVALID_ARG), (dict(n=-1), D.ERR_INVALID_ARG),
    (dict(n=5), D.ERR_INVALID_ARG), (dict(inter=2), D.ERR_INVALID_ARG), (dict(inverse=-1), D.ERR_INVALID_ARG),
    (dict(amp=math.nan), D.ERR_INVALID_ARG), (dict(freq=np.full(32, np.inf)), D.ERR_INVALID_ARG),
    (dict(freq=np.full(32, 1.5)), D.ERR_UNSUPPORTED), (dict(q=None), D.ERR_INVALID_ARG), (dict(v=F), D.ERR_INVALID_ARG),
    (dict(slot=F), D.ERR_INVALID_ARG),  # k in place through slots
    (dict(qos=(256, 64)), D.ERR_INVALID_ARG),  # q in place with other strides
])
def test_rotary_refusals(kw, code):
    assert _rotary(**kw) == code and D.load().dflash_last_error()


def test_rotary_nothing_to_do():
    assert _rotary(n=0) == 0


def _decode(n=2, hq=8, hkv=2, dh=64, pages=8, page=16, width=4, most=64, scale=0.0, window=0, dt=0, stride=4, qs=512, ws=256, q=F):
    return D.load().dflash_decode_attention_paged(q, qs, F, F, F, stride, F, n, hq, hkv, dh, pages, page, width, most, scale, window,
                                                  dt, F, None, ctypes.c_void_p(ws), 0, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dh=96), D.ERR_UNSUPPORTED), (dict(hq=7), D.ERR_INVALID_ARG), (dict(hkv=0), D.ERR_INVALID_ARG), (dict(n=-1), D.ERR_INVALID_ARG),
    (dict(page=0), D.ERR_INVALID_ARG), (dict(most=65), D.ERR_INVALID_ARG), (dict(window=-1), D.ERR_INVALID_ARG),
    (dict(scale=math.inf), D.ERR_INVALID_ARG), (dict(dt=2), D.ERR_INVALID_ARG), (dict(stride=3), D.ERR_INVALID_ARG),
    (dict(pages=0), D.ERR_INVALID_ARG), (dict(pages=1 << 28), D.ERR_UNSUPPORTED), (dict(qs=100), D.ERR_INVALID_ARG),
    (dict(n=1 << 20, width=1 << 13, stride=1 << 13, most=1 << 17), D.ERR_UNSUPPORTED), (dict(qs=504), D.ERR_INVALID_ARG), (dict(q=None), D.ERR_INVALID_ARG), (dict(ws=128), D.ERR_WORKSPACE),
])
def test_decode_refusals(kw, code):
    assert _decode(**kw) == code and D.load().dflash_last_error()


def test_decode_nothing_to_do():
    assert _decode(n=0) == 0


def _beam(n=2, w=4, k=4, vocab=100, eos=-1, dt=0, fin=None, ws=256, x=F):
    return D.load().dflash_beam_select(x, 400, 100, F, fin, n, w, k, vocab, eos, dt, ctypes.c_void_p(512), F, F, ctypes.c_void_p(512),
                                       ctypes.c_void_p(ws), 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(w=0), D.ERR_INVALID_ARG), (dict(k=0), D.ERR_INVALID_ARG), (dict(w=33), D.ERR_UNSUPPORTED), (dict(k=33), D.ERR_UNSUPPORTED),
    (dict(vocab=0), D.ERR_INVALID_ARG), (dict(eos=100), D.ERR_INVALID_ARG), (dict(eos=-2), D.ERR_INVALID_ARG), (dict(fin=F), D.ERR_INVALID_ARG),
    (dict(dt=5), D.ERR_INVALID_ARG), (dict(n=-1), D.ERR_INVALID_ARG), (dict(x=ctypes.c_void_p(257)), D.ERR_INVALID_ARG),
    (dict(ws=100), D.ERR_WORKSPACE), (dict(x=None), D.ERR_INVALID_ARG),
])
def test_beam_refusals(kw, code):
    assert _beam(**kw) == code and D.load().dflash_last_error()


def test_pages_refusals():
    lib = D.load()
    pools = (ctypes.c_void_p * 2)(256, 512)

    def fork(n=2, width=4, stride=4, pages=8):
        return lib.dflash_fork_pages(F, ctypes.c_void_p(512), F, stride, F, n, width, pages, None, None)

    assert fork(n=-1) == fork(stride=3) == fork(pages=-1) == D.ERR_INVALID_ARG
    assert fork(n=16385) == fork(pages=(1 << 30) + 1) == D.ERR_UNSUPPORTED
    assert fork(n=0) == 0
    assert lib.dflash_fork_pages(F, F, F, 4, F, 2, 4, 8, None, None) == D.ERR_INVALID_ARG  # parent is seq_lens

    def reserve(n_req=2, n=3, page=16, page_bytes=16 * 64, pools_=pools, count=2, pages=8, width=4, advance=0, ws=256):
        return lib.dflash_reserve_pages(F, F, F, width, F, pools_, count, page_bytes, n_req, n, width, page, pages, advance, F, F,
                                        ctypes.c_void_p(ws), 0, None, None)

    for kw in (dict(page=0), dict(n=-1), dict(page_bytes=0), dict(page_bytes=1000), dict(count=257), dict(count=-1), dict(advance=2),
               dict(pools_=None), dict(n_req=0), dict(pools_=(ctypes.c_void_p * 2)(256, 8))):
        assert reserve(**kw) == D.ERR_INVALID_ARG, kw
    assert reserve(pages=1 << 28) == reserve(width=1 << 28) == D.ERR_UNSUPPORTED
    assert reserve() == reserve(ws=100) == D.ERR_WORKSPACE
    assert reserve(n_req=0, n=0) == 0

    def compact(n=2, page_bytes=1024, used=F, ws=256, count=2):
        return lib.dflash_compact_pages(F, 4, F, pools, count, page_bytes, n, 4, 8, used, ctypes.c_void_p(ws), 0, None, None)

    assert compact(used=None) == compact(page_bytes=24) == compact(count=300) == D.ERR_INVALID_ARG
    assert compact() == D.ERR_WORKSPACE
    assert lib.dflash_pages_workspace_size(16385, 8) == 0 and lib.dflash_pages_workspace_size(4, 8) > 0


def test_frequency_tables():
    f, a = D.rotary_frequencies(8, 1e4)
    assert a == 1.0 and np.allclose(f, [1, 0.1, 0.01, 0.001])
    g, a = D.rotary_frequencies(8, 1e4, scaling="linear", factor=4.0)
    assert a == 1.0 and np.allclose(g * 4, f)
    g, a = D.rotary_frequencies(8, 1e4, scaling="base", factor=4.0)
    assert a == 1.0 and g[0] == 1.0 and np.isclose(g[-1] * 4, f[-1])
    g, a = D.rotary_frequencies(128, 1e4, scaling="parts", factor=4.0, original_len=4096)
    f, _ = D.rotary_frequencies(128, 1e4)
    turns = 4096 * f / (2 * math.pi)
    assert np.isclose(a, 0.1 * math.log(4.0) + 1.0)
    assert np.allclose(g[turns > 33], f[turns > 33]) and np.allclose(g[turns < 0.85] * 4, f[turns < 0.85])
    assert np.all(np.diff(g / f) <= 1e-15)
    for kw in (dict(rotary_dim=7), dict(theta=1.0), dict(factor=0.5), dict(scaling="x"), dict(scaling="parts"),
               dict(scaling="parts", original_len=10, fast=1.0, slow=2.0)):
        with pytest.raises(ValueError):
            D.rotary_frequencies(**{**dict(rotary_dim=8), **kw})


def test_bindings_refuse_what_is_no_cuda_tensor():
    import torch
    q, pos, f = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32), np.full(32, 0.5)
    with pytest.raises(ValueError):
        D.rotary(q, pos, f)
    with pytest.raises(ValueError):
        D.rotary(None, pos, f)
    with pytest.raises(TypeError):
        D.rotary([1.0], pos, f)
    with pytest.raises(ValueError):
        D.decode_attention_paged(q, q, q, pos, pos, max_ctx_len=4)
    with pytest.raises(ValueError):
        D.beam_select(q, q)
    with pytest.raises(TypeError):
        D.fork_pages(pos, pos, None, pos)
    with pytest.raises(ValueError):
        D.reserve_pages(pos, pos, q, pos, [], num_new=1)
    with pytest.raises(ValueError):
        D.compact_pages(q, pos, [])
    with pytest.raises(ValueError):
        D.rotary(q, pos, f, stream=0)
