"""The calls of a step over a shared prompt: host arguments that are refused before a device is touched, and the tables of
axes (CPU)."""
import ctypes
import math

import numpy as np
import pytest

import speculative_decoding_draft_rmsnorm_gb300 as D


def P(x):
    return ctypes.c_void_p(x)


def _norm(x=P(1 << 20), xs=64, r=None, rs=64, w=P(1 << 12), ro=None, ros=64, out=P(2 << 20), outs=64, scales=None, n=4, d=64, dt=0, wdt=0, odt=0, group=0,
          eps=1e-6):
    return D.load().dflash_rms_norm(x, xs, r, rs, w, ro, ros, out, outs, scales, n, d, dt, wdt, odt, group, eps, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), D.ERR_INVALID_ARG), (dict(wdt=2), D.ERR_INVALID_ARG), (dict(odt=3), D.ERR_INVALID_ARG), (dict(odt=1), D.ERR_UNSUPPORTED),
    (dict(n=-1), D.ERR_INVALID_ARG), (dict(d=0), D.ERR_INVALID_ARG), (dict(d=65537, xs=65537, outs=65537), D.ERR_UNSUPPORTED),
    (dict(eps=-1.0), D.ERR_INVALID_ARG), (dict(eps=math.nan), D.ERR_INVALID_ARG), (dict(eps=math.inf), D.ERR_INVALID_ARG),
    (dict(group=16), D.ERR_INVALID_ARG), (dict(odt=2, group=24, scales=P(4096)), D.ERR_INVALID_ARG), (dict(odt=2), D.ERR_INVALID_ARG),
    (dict(scales=P(4096)), D.ERR_INVALID_ARG), (dict(x=None), D.ERR_INVALID_ARG), (dict(r=P(3 << 20)), D.ERR_INVALID_ARG),
    (dict(ro=P(3 << 20)), D.ERR_INVALID_ARG), (dict(xs=-64), D.ERR_INVALID_ARG), (dict(outs=63), D.ERR_INVALID_ARG),
    (dict(x=P((1 << 20) + 1)), D.ERR_INVALID_ARG), (dict(out=P((1 << 20) + 64)), D.ERR_INVALID_ARG), (dict(out=P(1 << 20), outs=128), D.ERR_INVALID_ARG),
    (dict(w=P((2 << 20) + 128)), D.ERR_INVALID_ARG), (dict(odt=2, scales=P((1 << 20) + 64)), D.ERR_INVALID_ARG),
    (dict(odt=2, scales=P(4096), out=P(1 << 20)), D.ERR_INVALID_ARG),  # 8 bits over 16
    (dict(xs=200, outs=200, out=P((1 << 20) + 2 * 137)), D.ERR_INVALID_ARG),  # columns 137 .. 200 and 0 of the next row
])
def test_norm_refusals(kw, code):
    assert _norm(**kw) == code and D.load().dflash_last_error()


def test_norm_nothing_to_do():
    assert _norm(n=0) == 0


def _axes(n=4, axes=3, step=4, table=None, rd=64, pos=P(256), axis=0):
    f = np.full(rd // 2, 0.5)
    t = (ctypes.c_uint8 * (rd // 2))(*([axis] * (rd // 2))) if table is None else table
    F = P(1 << 20)
    return D.load().dflash_rotary_axes(F, 128, 64, F, 128, 64, 2, None, 0, 0, None, 0, 0, 0, None, 0, 0, None, 0, 0, pos, step, axes, t, None, n, n, 64, rd,
                                       f.ctypes.data, 1.0, 0, 0, 0, None, None)


@pytest.mark.parametrize("kw,code", [(dict(axes=0), D.ERR_INVALID_ARG), (dict(axes=-1), D.ERR_INVALID_ARG), (dict(axes=5), D.ERR_UNSUPPORTED),
                                     (dict(axis=3), D.ERR_INVALID_ARG), (dict(step=3), D.ERR_INVALID_ARG), (dict(rd=66), D.ERR_INVALID_ARG),
                                     (dict(pos=None), D.ERR_INVALID_ARG)])
def test_axes_refusals(kw, code):
    assert _axes(**kw) == code and D.load().dflash_last_error()


def test_axes_nothing_to_do():
    assert _axes(n=0) == 0


def _prefixes(n=4, groups=2, width=8, stride=8, page=16, table=P(4096), lens=P(8192), starts=P(12288), out=P(16384)):
    return D.load().dflash_shared_prefixes(table, stride, lens, starts, n, groups, width, page, out, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=-1), D.ERR_INVALID_ARG), (dict(groups=-1), D.ERR_INVALID_ARG), (dict(width=-1), D.ERR_INVALID_ARG), (dict(page=0), D.ERR_INVALID_ARG),
    (dict(stride=7), D.ERR_INVALID_ARG), (dict(groups=(1 << 24) + 1), D.ERR_UNSUPPORTED), (dict(out=None), D.ERR_INVALID_ARG),
    (dict(lens=None), D.ERR_INVALID_ARG), (dict(table=None), D.ERR_INVALID_ARG), (dict(out=P(8192 + 12)), D.ERR_INVALID_ARG),
    (dict(out=P(12288 + 8)), D.ERR_INVALID_ARG), (dict(out=P(4096 + 124)), D.ERR_INVALID_ARG),
])
def test_prefix_refusals(kw, code):
    assert _prefixes(**kw) == code and D.load().dflash_last_error()


def test_prefixes_nothing_to_do():
    assert _prefixes(groups=0) == 0


def test_tables_of_axes():
    assert D.rotary_sections((2, 0, 3)).tolist() == [0, 0, 2, 2, 2]
    assert D.rotary_sections((3, 1, 2), interleaved=True).tolist() == [0, 1, 2, 0, 2, 0]
    assert D.rotary_sections([4]).dtype == np.uint8
    for bad in ((), (1, -1), range(300)):
        with pytest.raises(ValueError):
            D.rotary_sections(bad)


def test_bindings_refuse_what_is_no_cuda_tensor():
    import torch
    x, i, f = torch.zeros(2, 64), torch.zeros(2, dtype=torch.int32), np.full(32, 0.5)
    for call in (lambda: D.rms_norm(x, x[0]), lambda: D.rms_norm([1.0], x), lambda: D.rms_norm(x, x[0], stream=0),
                 lambda: D.rotary_axes(x.view(2, 1, 64), i.view(1, 2), [0] * 32, f), lambda: D.rotary_axes(None, i, [0], f),
                 lambda: D.shared_prefixes(i.view(1, 2), i, i, page_size=16), lambda: D.shared_prefixes(None, i, i, page_size=16)):
        with pytest.raises((TypeError, ValueError)):
            call()


def _shared(n=2, groups=1, hq=8, hkv=2, dh=64, pages=8, page=16, width=4, most=64, scale=0.0, window=0, dt=0, stride=4, qs=512, ws=256, q=P(1 << 20),
            starts=P(4096), prefixes=P(8192), flags=0):
    F = P(1 << 20)
    return D.load().dflash_decode_attention_shared(q, qs, F, F, F, stride, F, starts, prefixes, n, groups, hq, hkv, dh, pages, page, width, most, scale, window,
                                                   dt, F, None, P(ws), 0, flags, None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dh=96), D.ERR_UNSUPPORTED), (dict(hq=7), D.ERR_INVALID_ARG), (dict(hkv=0), D.ERR_INVALID_ARG), (dict(n=-1), D.ERR_INVALID_ARG),
    (dict(groups=-1), D.ERR_INVALID_ARG), (dict(groups=(1 << 24) + 1), D.ERR_UNSUPPORTED), (dict(starts=None), D.ERR_INVALID_ARG),
    (dict(prefixes=None), D.ERR_INVALID_ARG), (dict(page=0), D.ERR_INVALID_ARG), (dict(most=65), D.ERR_INVALID_ARG),
    (dict(window=-1), D.ERR_INVALID_ARG), (dict(scale=math.inf), D.ERR_INVALID_ARG), (dict(dt=2), D.ERR_INVALID_ARG),
    (dict(stride=3), D.ERR_INVALID_ARG), (dict(pages=0), D.ERR_INVALID_ARG), (dict(qs=100), D.ERR_INVALID_ARG), (dict(q=None), D.ERR_INVALID_ARG),
    (dict(ws=128), D.ERR_WORKSPACE), (dict(flags=1), D.ERR_INVALID_ARG), (dict(flags=6), D.ERR_INVALID_ARG),
])
def test_shared_refusals(kw, code):
    assert _shared(**kw) == code and D.load().dflash_last_error()


def test_shared_nothing_to_do():
    assert _shared(n=0) == 0
