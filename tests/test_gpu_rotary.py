"""dflash_rotary on the GPU against the definition in 64 bits.

Tolerance, relative to a (|u| + |v|) of an element's pair: the angle in turns is rounded twice at
magnitude <= 1 (2^-24 turns = 3.8e-7 rad), sine and cosine carry 2^-23, the amplitude and the two
products 2^-24 each: below 1e-6. A bf16 output adds half a step, 2^-8 of its value.
"""
import numpy as np
import pytest

from tests import decode_ref as R

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def check(got, x, pos, freq, **kw):
    import torch
    want, size = R.rotary(x.double().cpu().numpy(), pos.cpu().numpy(), freq, **kw)
    tol = 1e-6 * size + (2.0 ** -8 * np.abs(want) if got.dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


def inputs(n, hq, hkv, dh, dtype, seed=0, far=32768):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(n, hq + 2 * hkv, dh, device="cuda", generator=g).to(dtype)
    pos = torch.randint(0, far, (n,), device="cuda", generator=g, dtype=torch.int32)
    return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,hq,hkv,dh,rd", [(1, 1, 1, 64, 64), (3, 32, 8, 128, 128), (129, 4, 2, 80, 20), (7, 5, 1, 96, 90),
                                            (33, 16, 4, 256, 256), (2, 3, 3, 6, 2), (500, 8, 2, 128, 64), (5, 2, 1, 72, 36)])
def test_matches_definition(inter, f32, n, hq, hkv, dh, rd):
    import torch
    q, k, _, pos = inputs(n, hq, hkv, dh, torch.float32 if f32 else torch.bfloat16)
    freq, _ = D().rotary_frequencies(rd)
    gq, gk = D().rotary(q, pos, freq, k=k, interleaved=inter)
    check(gq, q, pos, freq, interleaved=inter)
    check(gk, k, pos, freq, interleaved=inter)
    assert torch.equal(gq[..., rd:], q[..., rd:]) and torch.equal(gk[..., rd:], k[..., rd:])


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "parts"])
def test_scaled_frequencies_and_far_positions(scaling):
    import torch
    q, k, _, pos = inputs(64, 4, 2, 128, torch.float32, far=1 << 24)
    pos[0], pos[1], pos[2] = 0, (1 << 24) - 1, -5
    freq, amp = D().rotary_frequencies(128, 1e4, scaling=scaling, factor=8.0, original_len=4096)
    gq, gk = D().rotary(q, pos, freq, k=k, amplitude=amp)
    check(gq, q, pos, freq, amplitude=amp)
    check(gk, k, pos, freq, amplitude=amp)


@pytest.mark.parametrize("off", [0, 1, 2, 3])
@pytest.mark.parametrize("f32", [False, True])
def test_strides_alignment_and_in_place(off, f32):
    import torch
    dt = torch.float32 if f32 else torch.bfloat16
    base = torch.randn(11, 7, 140, device="cuda").to(dt)
    q, k = base[:, 1:5, off:off + 128], base[:, 5:7, off:off + 128]
    keep = base.clone()
    pos = torch.arange(11, device="cuda", dtype=torch.int32) * 97
    freq, _ = D().rotary_frequencies(128)
    want, _ = D().rotary(keep[:, 1:5, off:off + 128].contiguous(), pos, freq)
    wk, _ = D().rotary(keep[:, 5:7, off:off + 128].contiguous(), pos, freq)
    D().rotary(q, pos, freq, k=k, q_out=q, k_out=k)
    assert torch.equal(q, want) and torch.equal(k, wk)  # the same arithmetic whatever the access width
    untouched = torch.ones(7, 140, dtype=torch.bool, device="cuda")
    untouched[1:7, off:off + 128] = False
    assert torch.equal(base[:, untouched], keep[:, untouched])
    part, _ = D().rotary_frequencies(32)
    a = keep[:, 1:5, off:off + 128]
    w2, _ = D().rotary(a, pos, part, interleaved=True)
    D().rotary(a, pos, part, interleaved=True, q_out=a)
    assert torch.equal(a, w2)


def test_store_slots_padding_and_status():
    import torch
    n, hkv, dh = 21, 4, 128
    q, k, v, pos = inputs(n, 8, hkv, dh, torch.bfloat16, seed=3)
    freq, _ = D().rotary_frequencies(dh)
    pool_k = torch.full((9, 5, hkv, dh), 7.0, device="cuda", dtype=torch.bfloat16)
    pool_v = pool_k.clone()
    slot = torch.randperm(45, device="cuda")[:n].to(torch.int32)
    slot[4], slot[9] = -1, 45  # padding; out of range
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gq, _ = D().rotary(q, pos, freq, k=k, k_out=pool_k, v=v, v_out=pool_v, slot=slot, status=status)
    _, dense = D().rotary(None, pos, freq, k=k)
    check(gq, q, pos, freq)
    want_k, want_v = torch.full((45, hkv, dh), 7.0, device="cuda", dtype=torch.bfloat16), None
    want_v = want_k.clone()
    ok = (slot >= 0) & (slot < 45)
    want_k[slot[ok].long()], want_v[slot[ok].long()] = dense[ok], v[ok]
    assert torch.equal(pool_k.view(45, hkv, dh), want_k) and torch.equal(pool_v.view(45, hkv, dh), want_v)
    assert status.item() == D().STATUS_METADATA
    status.zero_()
    slot[9] = -1
    D().rotary(q, pos, freq, k=k, k_out=pool_k, slot=slot, status=status)
    assert status.item() == 0


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_is_the_gradient(inter):
    # L = <w, f(x)> has the gradient f^T w: by the formula, and by differences (f is linear, so a
    # difference is exact up to its rounding)
    import torch
    n, h, dh, rd = 6, 3, 16, 12
    x, _, _, pos = inputs(n, h, 1, dh, torch.float32, seed=5)
    w = torch.randn(n, h, dh, device="cuda")
    freq, amp = D().rotary_frequencies(rd, scaling="parts", factor=4.0, original_len=4096)
    grad, _ = D().rotary(w, pos, freq, amplitude=amp, interleaved=inter, inverse=True)
    check(grad, w, pos, freq, amplitude=amp, interleaved=inter, inverse=True)
    x = x.contiguous()
    for t, i, d in [(0, 0, 0), (1, 2, 11), (2, 1, 12), (5, 0, 7), (3, 2, 15)]:
        lo, hi = x.clone(), x.clone()
        lo[t, i, d] -= 1.0
        hi[t, i, d] += 1.0
        f = lambda y: (w.double() * D().rotary(y, pos, freq, amplitude=amp, interleaved=inter)[0].double()).sum().item()  # noqa: E731
        # both evaluations round dh outputs of size <= a (|u| + |v|) <= 12 by 2e-6 of it
        assert abs((f(hi) - f(lo)) / 2 - grad[t, i, d].item()) < n * h * dh * 12 * 4 * 2e-6


def test_rotation_then_inverse_and_zero_rows():
    import torch
    q, _, _, pos = inputs(0, 4, 1, 64, torch.float32)
    freq, _ = D().rotary_frequencies(64)
    out, _ = D().rotary(q, pos, freq)
    assert out.shape == (0, 4, 64)
    q, _, _, pos = inputs(40, 4, 1, 64, torch.float32)
    back, _ = D().rotary(D().rotary(q, pos, freq)[0], pos, freq, inverse=True)
    size = R.rotary(q.double().cpu().numpy(), pos.cpu().numpy(), freq)[1]
    assert np.all(np.abs((back - q).double().cpu().numpy()) <= 4e-6 * size)  # two passes, pairs of pairs


def test_stream_and_graph():
    import torch
    q, k, v, pos = inputs(9, 4, 2, 128, torch.bfloat16, seed=8)
    freq, _ = D().rotary_frequencies(128)
    want, wk = D().rotary(q, pos, freq, k=k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = D().rotary(q, pos, freq, k=k, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    qo, ko = torch.empty_like(want), torch.empty_like(wk)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D().rotary(q, pos, freq, k=k, q_out=qo, k_out=ko)
    pos += 11
    g.replay()
    want, wk = D().rotary(q, pos, freq, k=k)
    assert torch.equal(qo, want) and torch.equal(ko, wk)


def test_refusals():
    import torch
    q, k, v, pos = inputs(4, 4, 2, 64, torch.bfloat16)
    freq, _ = D().rotary_frequencies(64)
    d = D()
    with pytest.raises(TypeError):
        d.rotary(q.half(), pos, freq)
    with pytest.raises(TypeError):
        d.rotary(q, pos.long(), freq)
    with pytest.raises(TypeError):
        d.rotary(q, pos, freq, k=k.float())
    with pytest.raises(ValueError):
        d.rotary(q, pos[:3], freq)
    with pytest.raises(ValueError):
        d.rotary(q.transpose(1, 2), pos, freq)
    with pytest.raises(ValueError):
        d.rotary(q, pos, freq, v=v)
    with pytest.raises(ValueError):
        d.rotary(q, pos, freq, k=k, slot=pos)  # slots need a destination
    with pytest.raises(ValueError):
        d.rotary(q.cpu(), pos, freq)
    big, _ = d.rotary_frequencies(66)
    for bad in (big, freq * 100.0, freq * np.nan):
        with pytest.raises(d.DFlashError):
            d.rotary(q, pos, bad)
    with pytest.raises(d.DFlashError):
        d.rotary(q, pos, freq, amplitude=float("inf"))
    with pytest.raises(d.DFlashError):  # in place through slots
        kk = k.contiguous()
        d.rotary(q, pos, freq, k=kk, k_out=kk, slot=pos)
