"""dflash_rms_norm on the GPU against the definition in 64 bits.

Tolerance: a thread adds at most 80 squares, and 10 more additions join the block's, all of positive terms: the sum is
within 90 x 2^-24, its root within half of that; the mean, eps, root, quotient and three products add 2^-24 each:
64 x 2^-24 together, relative to y. An output adds half a step of its type: 2^-8 (bf16), 2^-24 (f32), 2^-4 (e4m3; half of its
least step, 2^-10, below 2^-6). A scale is such a y, divided once more.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu
TOL = 64 * 2.0 ** -24


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def inputs(n, d, f32, w32=False, seed=0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = torch.float32 if f32 else torch.bfloat16
    x = torch.randn(n, d, device="cuda", generator=g).to(dt)
    r = (5 * torch.randn(n, d, device="cuda", generator=g)).to(dt)
    w = (1 + 0.3 * torch.randn(d, device="cuda", generator=g)).to(torch.float32 if w32 else torch.bfloat16)
    return x, r, w


def check(got, x, r, w, group=0, eps=1e-6):
    import torch
    out, stream, scales = got
    h = x.double()
    if r is not None:
        s = x.double() + r.double()
        half = torch.finfo(x.dtype).eps / 2
        assert bool(((stream.double() - s).abs() <= (half + 2.0 ** -24) * s.abs()).all())
        h = stream.double()
    else:
        assert stream is None
    y = h * w.double() / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    if out.dtype != torch.float8_e4m3fn:
        assert scales is None and out.dtype == x.dtype
        assert bool(((out.double() - y).abs() <= (torch.finfo(out.dtype).eps / 2 + TOL) * y.abs()).all())
        return
    n, d = x.shape
    each = group or d
    parts = y.split(each, 1)
    assert scales.shape == (n, len(parts)) and scales.dtype == torch.float32
    want = torch.stack([(p.abs().amax(1) / 448).clamp(min=2.0 ** -126) for p in parts], 1)
    assert bool(((scales.double() - want).abs() <= (TOL + 2.0 ** -24) * want).all())
    v = y / scales.double().repeat_interleave(each, 1)[:, :d]
    step = torch.maximum(2.0 ** -4 * v.abs(), torch.full_like(v, 2.0 ** -10))
    assert bool(((out.double() - v).abs() <= step + (TOL + 2.0 ** -23) * v.abs()).all())


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,d", [(1, 1), (3, 2), (2, 7), (5, 16), (4, 64), (3, 130), (1, 2560), (7, 1000), (33, 5003), (2, 5120), (300, 256),
                                 (3, 16384), (2, 20001), (2, 40002), (1, 65536)])
def test_matches_definition(n, d, f32, residual):
    x, r, w = inputs(n, d, f32, w32=f32, seed=d)
    check(D().rms_norm(x, w, residual=r if residual else None), x, r if residual else None, w)


@pytest.mark.parametrize("f32,w32", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("n,d,group", [(1, 2560, 0), (3, 7, 0), (2, 40002, 0), (65, 1024, 0), (1, 5120, 128), (9, 5120, 64), (3, 1000, 128), (2, 5003, 128),
                                       (4, 130, 16), (4, 130, 48), (2, 4096, 4096), (2, 4096, 512), (3, 100, 128), (2, 24000, 128),
                                       (2, 65536, 16), (5, 96, 32), (2, 4097, 32)])
def test_eight_bits(n, d, group, f32, w32):
    x, r, w = inputs(n, d, f32, w32, seed=d + group)
    check(D().rms_norm(x, w, residual=r, out_dtype=D().OUT_E4M3, group_size=group), x, r, w, group)
    check(D().rms_norm(x, w, out_dtype=D().OUT_E4M3, group_size=group, eps=0.1), x, None, w, group, eps=0.1)


@pytest.mark.parametrize("eight,group", [(False, 0), (True, 0), (True, 128), (True, 48)])
def test_zeros_nans_infinities_and_small_rows(eight, group):
    import torch
    x, _, w = inputs(6, 640, False)
    x[0] = 0
    x[1, 5] = float("nan")
    x[2, 600] = float("inf")
    x[3] *= 2.0 ** -100
    x[4, 100] = 300.0
    kw = dict(out_dtype=D().OUT_E4M3, group_size=group) if eight else {}
    out, _, scales = D().rms_norm(x, w, **kw)
    whole, _, ws = D().rms_norm(x[3:], w, **kw)
    assert torch.equal(out[3:].view(torch.uint8), whole.view(torch.uint8))  # rows do not touch one another
    check((whole, None, ws), x[3:], None, w, group)
    value = out.float() * (scales.repeat_interleave(group or 640, 1)[:, :640] if eight else 1)
    assert not value[0].any() and bool(value[1].isnan().all()) and bool(value[2, 600].isnan()) and bool((value[2].isnan() | (value[2] == 0)).all())
    if eight:
        assert bool((scales[0] == 2.0 ** -126).all()) and bool(scales[1].isnan().all())


@pytest.mark.parametrize("off", [0, 1, 2, 4, 8])
@pytest.mark.parametrize("f32", [False, True])
def test_strides_alignment_and_in_place(off, f32):
    import torch
    n, d = 11, 640
    x, r, w = inputs(n, d, f32)
    base = torch.zeros(n, 2 * d + 48, device="cuda", dtype=x.dtype)
    xs, rs = base[:, off:off + d], base[:, d + 16 + off:2 * d + 16 + off]
    xs.copy_(x), rs.copy_(r)
    want = D().rms_norm(x, w, residual=r)
    q = D().rms_norm(x, w, residual=r, out_dtype=D().OUT_E4M3, group_size=64)
    got = D().rms_norm(xs, w, residual=rs, out_dtype=D().OUT_E4M3, group_size=64)
    # another access width adds a row's squares in another order
    assert bool(((got[2] - q[2]).abs() <= 2 * TOL * q[2]).all()) and torch.equal(got[1], q[1])
    check(got, xs, rs, w, 64)
    keep = base.clone()
    out, stream, _ = D().rms_norm(xs, w, residual=rs, residual_out=rs, out=xs)  # both in place
    assert out is xs and stream is rs and torch.equal(rs, want[1])
    check((xs, rs, None), x, r, w)
    untouched = torch.ones(base.shape[1], dtype=torch.bool, device="cuda")
    untouched[off:off + d] = untouched[d + 16 + off:2 * d + 16 + off] = False
    assert torch.equal(base[:, untouched], keep[:, untouched])
    # the stream over the layer's output, the norm over the old stream
    y, s = x.clone(), r.clone()
    D().rms_norm(y, w, residual=s, residual_out=y, out=s)
    assert torch.equal(y, want[1]) and torch.equal(s, want[0])
    got = D().rms_norm(x[:1].expand(n, d), w, residual=r)  # one row for all
    check(got, x[:1].expand(n, d), r, w)


def test_long_rows_in_place():
    import torch
    x, r, w = inputs(2, 60000, True)
    want = D().rms_norm(x, w, residual=r)
    y, s = x.clone(), r.clone()
    D().rms_norm(y, w, residual=s, residual_out=s, out=y)
    assert torch.equal(y, want[0]) and torch.equal(s, want[1])
    y = x.clone()
    D().rms_norm(y, w, out=y)
    assert torch.equal(y, D().rms_norm(x, w)[0])


def test_refusals():
    import torch
    lib = D()
    x, r, w = inputs(4, 64, False)
    for kw in (dict(group_size=64), dict(out_dtype=lib.OUT_F32), dict(out_dtype=lib.OUT_E4M3, group_size=24), dict(residual=r[:3]), dict(residual=r.float()),
               dict(residual_out=r), dict(scales=torch.zeros(4, 1, device="cuda")), dict(out=torch.zeros(4, 64, device="cuda")),
               dict(out_dtype=7), dict(residual=r.cpu()), dict(out_dtype=lib.OUT_E4M3, scales=torch.zeros(4, 2, device="cuda")),
               dict(eps="x"), dict(residual=[1.0]), dict(out=x.t()[:4])):
        with pytest.raises((TypeError, ValueError)):
            lib.rms_norm(x, w, **kw)
    wide = torch.zeros(4, 100, device="cuda", dtype=torch.bfloat16)
    for kw in (dict(eps=-1.0), dict(eps=float("nan")), dict(residual=r, residual_out=x, out=x), dict(out=wide[:, :64], residual=wide[:, 30:94]),
               dict(out=x[:1].expand(4, 64)), dict(residual=r, residual_out=wide[:, 36:], out=wide[:, :64])):
        with pytest.raises(lib.DFlashError):
            lib.rms_norm(x, w, **kw)
    with pytest.raises(lib.DFlashError):
        lib.rms_norm(torch.zeros(1, 65537, device="cuda"), torch.zeros(65537, device="cuda"))
    for bad in ((x.half(), w), (x, w.half()), (x, w[:63]), (x[0], w), (x.cpu(), w), (x, w.cpu())):
        with pytest.raises((TypeError, ValueError)):
            lib.rms_norm(*bad)
    for t in (x, w):
        t.requires_grad_(True)
        with pytest.raises(ValueError):
            lib.rms_norm(x, w)
        with torch.no_grad():
            lib.rms_norm(x, w)
        t.requires_grad_(False)
    both = torch.zeros(4, 128, device="cuda", dtype=torch.bfloat16)
    both[:, 64:] = x
    check((lib.rms_norm(both[:, 64:], w, out=both[:, :64])[0], None, None), x, None, w)  # side by side in one buffer


def test_no_rows_streams_versions_and_graphs():
    import torch
    x, r, w = inputs(0, 64, False)
    out, s, scales = D().rms_norm(x, w, residual=r, out_dtype=D().OUT_E4M3)
    assert out.shape == s.shape == (0, 64) and scales.shape == (0, 1)
    x, r, w = inputs(50, 4096, False)
    want = D().rms_norm(x, w, residual=r)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = D().rms_norm(x, w, residual=r, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:2], want))
    out, v = torch.empty_like(x), r._version
    D().rms_norm(x, w, residual=r.clone(), out=out)
    assert out._version == 1 and r._version == v
    g = torch.cuda.CUDAGraph()
    stream = r.clone()
    with torch.cuda.graph(g):
        D().rms_norm(x, w, residual=stream, residual_out=stream, out=out)
    stream.copy_(r)
    g.replay()
    assert torch.equal(out, want[0]) and torch.equal(stream, want[1])
    g.replay()
    assert torch.equal(stream, (want[1].float() + x.float()).to(torch.bfloat16))


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("f32,d", [(False, 5120), (False, 256), (False, 8192), (False, 16384), (False, 1032), (True, 4096), (True, 128), (True, 12000)])
@pytest.mark.parametrize("eight,group", [(False, 0), (True, 0), (True, 128), (True, 16), (True, 80)])
def test_many_rows(f32, d, eight, group, residual):
    import torch
    n = 3001
    x, r, w = inputs(n, d, f32, seed=d + group)
    kw = dict(out_dtype=D().OUT_E4M3, group_size=group) if eight else {}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = D().rms_norm(x, w, residual=r if residual else None, status=status, **kw)
    check(got, x, r if residual else None, w, group)
    assert status.item() == 0
    y, s = x.clone(), r.clone()  # in place
    out, stream, _ = D().rms_norm(y, w, residual=s, residual_out=s, out=None if eight else y, **kw)
    check((out, stream, _), x, r, w, group)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("d", [33, 65, 127, 1001, 2562, 5003, 8191, 8193, 16383, 16385])
@pytest.mark.parametrize("eight,group", [(False, 0), (True, 0), (True, 16), (True, 112), (True, 128)])
def test_odd_widths(d, f32, eight, group, residual):
    import torch
    n = 37
    x, r, w = inputs(n, d, f32, w32=d % 4 == 1, seed=d + group)
    kw = dict(out_dtype=D().OUT_E4M3, group_size=group) if eight else {}
    check(D().rms_norm(x, w, residual=r if residual else None, **kw), x, r if residual else None, w, group)
    y, s = x.clone(), r.clone()  # in place
    out, stream, _ = D().rms_norm(y, w, residual=s, residual_out=s, out=None if eight else y, **kw)
    check((out, stream, _), x, r, w, group)
    wide = torch.zeros(n, d + 8, device="cuda", dtype=x.dtype)  # rows that lie elsewhere in the stream than in x
    out, stream, _ = D().rms_norm(x, w, residual=r, residual_out=wide[:, 3:3 + d], **kw)
    check((out, stream, _), x, r, w, group)
    assert not wide[:, :3].any() and not wide[:, 3 + d:].any()
    out, stream, _ = D().rms_norm(x[:1].expand(n, d), w, residual=r, **kw)
    check((out, stream, _), x[:1].expand(n, d), r, w, group)


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("group", [None, 0, 16, 48, 64, 128])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,d", [(5003, 17), (4870, 50), (5001, 97), (4999, 100), (5000, 129), (4900, 257), (4867, 511), (5001, 640), (5003, 16), (5001, 64),
                                 (4999, 128), (5000, 200), (4990, 256), (700, 33), (33, 127), (1, 65), (9, 250)])
def test_narrow_rows(n, d, f32, group, residual):
    import torch
    x, r, w = inputs(n, d, f32, w32=d % 2 == 0, seed=d)
    kw = {} if group is None else dict(out_dtype=D().OUT_E4M3, group_size=group)
    res = r if residual else None
    got = D().rms_norm(x, w, residual=res, **kw)
    check(got, x, res, w, group or 0)
    # the same rows, far apart and out of step with memory's alignment: the same values to within the order of their sums
    wide = torch.zeros(n, d + 37, device="cuda", dtype=x.dtype)
    wide[:, 5:5 + d] = x
    check(D().rms_norm(wide[:, 5:5 + d], w, residual=res, **kw), x, res, w, group or 0)
    wide = torch.zeros(n, (d + 23) // 8 * 8, device="cuda", dtype=x.dtype)  # aligned and apart
    wide[:, :d] = x
    check(D().rms_norm(wide[:, :d], w, residual=res, **kw), x, res, w, group or 0)
    if residual:  # in place
        x1, r1 = x.clone(), r.clone()
        same = D().rms_norm(x1, w, residual=r1, residual_out=x1, **kw)
        assert torch.equal(same[0].float(), got[0].float()) and torch.equal(x1, got[1]) and torch.equal(r1, r)


@pytest.mark.parametrize("d", [17, 64, 130])
@pytest.mark.parametrize("eight", [False, True])
def test_narrow_rows_of_zeros_nans_and_infinities(d, eight):
    import torch
    n = 6000
    x, _, w = inputs(n, d, False, seed=d)
    kw = dict(out_dtype=D().OUT_E4M3) if eight else {}
    want = D().rms_norm(x, w, **kw)
    x[1::7], x[2::7, 3], x[3::7, 1] = 0.0, float("nan"), float("inf")
    got = D().rms_norm(x, w, **kw)
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[1::7] = rest[2::7] = rest[3::7] = False
    assert torch.equal(got[0].float()[rest], want[0].float()[rest])
    assert bool((got[0].float()[1::7] == 0).all())
    assert bool(torch.isnan(got[0].float()[2::7]).all())
    if eight:
        assert torch.equal(got[2][rest], want[2][rest]) and bool((got[2][1::7] == 2.0 ** -126).all()) and bool(torch.isnan(got[2][2::7]).all())
