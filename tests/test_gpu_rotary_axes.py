"""dflash_rotary_axes on the GPU against the definition in 64 bits; tolerances are those of dflash_rotary's tests."""
import numpy as np
import pytest

from tests import test_gpu_rotary as T

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def check(got, x, pos, axes, freq, amplitude=1.0, interleaved=False, inverse=False):
    """By the definition: pair after pair, with its own axis's positions."""
    import torch
    x, pos = x.double().cpu().numpy(), pos.cpu().numpy().astype(np.float64)
    pairs = len(freq)
    want, size = x.copy(), np.zeros_like(x)
    for i in range(pairs):
        u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        t = (pos[axes[i]] * freq[i])[:, None]
        s = np.sin(-t if inverse else t)
        want[..., u] = amplitude * (x[..., u] * np.cos(t) - x[..., v] * s)
        want[..., v] = amplitude * (x[..., v] * np.cos(t) + x[..., u] * s)
        size[..., u] = size[..., v] = abs(amplitude) * (np.abs(x[..., u]) + np.abs(x[..., v]))
    tol = 1e-6 * size + (2.0 ** -8 * np.abs(want) if got.dtype == torch.bfloat16 else 0.0)
    assert np.all(np.abs(got.double().cpu().numpy() - want) <= tol)


def positions(axes, n, seed=0, far=40000):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(-far // 8, far, (axes, n), device="cuda", generator=g, dtype=torch.int32)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,hq,hkv,dh,sections", [(1, 1, 1, 64, (32,)), (3, 32, 8, 128, (16, 24, 24)), (129, 4, 2, 80, (3, 7)), (7, 5, 1, 96, (1, 2, 3, 39)),
                                                  (33, 16, 4, 256, (0, 64, 64)), (2, 3, 3, 6, (1,)), (300, 8, 2, 128, (8, 12, 12)),
                                                  (5, 2, 1, 72, (9, 9))])
def test_matches_definition(n, hq, hkv, dh, sections, f32, inter, inverse):
    import torch
    q, k, _, _ = T.inputs(n, hq, hkv, dh, torch.float32 if f32 else torch.bfloat16)
    rd = 2 * sum(sections)
    freq, _ = D().rotary_frequencies(rd)
    pos = positions(len(sections), n)
    for dealt in (False, True):
        axes = D().rotary_sections(sections, interleaved=dealt)
        gq, gk = D().rotary_axes(q, pos, axes, freq, k=k, interleaved=inter, inverse=inverse, amplitude=1.25)
        check(gq, q, pos, axes, freq, 1.25, inter, inverse)
        check(gk, k, pos, axes, freq, 1.25, inter, inverse)
        assert torch.equal(gq[..., rd:], q[..., rd:]) and torch.equal(gk[..., rd:], k[..., rd:])


def test_equal_axes_are_one():
    # the same bits as with one position a token
    import torch
    q, k, _, pos = T.inputs(77, 8, 2, 128, torch.bfloat16)
    freq, amp = D().rotary_frequencies(128, scaling="parts", factor=4.0, original_len=4096)
    want = D().rotary(q, pos, freq, k=k, amplitude=amp)
    got = D().rotary_axes(q, pos.expand(3, 77).contiguous(), D().rotary_sections((16, 24, 24)), freq, k=k, amplitude=amp)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_store_strides_lists_and_in_place():
    import torch
    n, hkv, dh = 21, 4, 128
    q, k, v, _ = T.inputs(n, 8, hkv, dh, torch.bfloat16, seed=3)
    freq, _ = D().rotary_frequencies(dh)
    axes = D().rotary_sections((16, 24, 24))
    pos = positions(3, n + 5)[:, :n]  # rows of a wider tensor
    want_q, want_k = D().rotary_axes(q, pos.contiguous(), axes, freq, k=k)
    pool_k = torch.full((9, 5, hkv, dh), 7.0, device="cuda", dtype=torch.bfloat16)
    pool_v = pool_k.clone()
    slot = torch.randperm(45, device="cuda")[:n].to(torch.int32)
    slot[4], slot[9] = -1, 45
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gq, _ = D().rotary_axes(q, pos, axes.tolist(), freq, k=k, k_out=pool_k, v=v, v_out=pool_v, slot=slot, status=status)
    assert torch.equal(gq, want_q) and status.item() == D().STATUS_METADATA
    kk = torch.full((45, hkv, dh), 7.0, device="cuda", dtype=torch.bfloat16)
    vv = kk.clone()
    ok = (slot >= 0) & (slot < 45)
    kk[slot[ok].long()], vv[slot[ok].long()] = want_k[ok], v[ok]
    assert torch.equal(pool_k.view(45, hkv, dh), kk) and torch.equal(pool_v.view(45, hkv, dh), vv)
    D().rotary_axes(q, pos, axes.astype(np.int64), freq, k=k, q_out=q, k_out=k)
    assert torch.equal(q, want_q) and torch.equal(k, want_k)


@pytest.mark.parametrize("inter", [False, True])
def test_inverse_is_the_gradient(inter):
    # as for one axis: by differences (the map is linear, so a difference is exact up to its rounding)
    import torch
    n, h, dh = 6, 3, 16
    x, _, _, _ = T.inputs(n, h, 1, dh, torch.float32, seed=5)
    x, w, pos = x.contiguous(), torch.randn(n, h, dh, device="cuda"), positions(3, n)
    freq, _ = D().rotary_frequencies(12)
    axes = D().rotary_sections((1, 3, 2), interleaved=True)
    grad, _ = D().rotary_axes(w, pos, axes, freq, interleaved=inter, inverse=True)
    for t, i, d in [(0, 0, 0), (1, 2, 11), (2, 1, 12), (5, 0, 7), (3, 2, 15)]:
        lo, hi = x.clone(), x.clone()
        lo[t, i, d] -= 1.0
        hi[t, i, d] += 1.0
        f = lambda y: (w.double() * D().rotary_axes(y, pos, axes, freq, interleaved=inter)[0].double()).sum().item()  # noqa: E731
        assert abs((f(hi) - f(lo)) / 2 - grad[t, i, d].item()) < n * h * dh * 12 * 4 * 2e-6


def test_refusals_no_rows_and_capture():
    import torch
    lib = D()
    q, k, _, _ = T.inputs(9, 4, 2, 64, torch.bfloat16)
    freq, _ = lib.rotary_frequencies(64)
    axes, pos = lib.rotary_sections((16, 16)), positions(2, 9)
    for p, a in ((pos[0], axes), (pos[:, :8], axes), (pos.long(), axes), (pos, axes[:31]), (pos, axes.astype(np.float32)), (pos, [300] * 32),
                 (pos, [-1] * 32), (pos.t().contiguous().t(), axes), (pos.cpu(), axes)):
        with pytest.raises((TypeError, ValueError)):
            lib.rotary_axes(q, p, a, freq)
    for p, a in ((pos, [2] * 32), (positions(5, 9), axes), (pos[:1].expand(2, 9), axes), (positions(0, 9), axes)):
        with pytest.raises(lib.DFlashError):
            lib.rotary_axes(q, p, a, freq)
    with pytest.raises(ValueError):
        lib.rotary_axes(q.float().requires_grad_(True), pos, axes, freq)
    e, _ = lib.rotary_axes(q[:0], pos[:, :0], axes, freq)
    assert e.shape == (0, 4, 64)
    want, _ = lib.rotary_axes(q, pos + 3, axes, freq)
    out, g = torch.empty_like(want), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.rotary_axes(q, pos, axes, freq, q_out=out)
    pos += 3
    g.replay()
    assert torch.equal(out, want)
