"""Bounded device waits of the step over a shared prompt that run out, and the calls after them.

As in test_gpu_wait_timeout.py: the test library is the product's sources built with DFLASH_WAIT_TEST, where a wait gives up
after 5 ms and a hook withholds one copy, so that the wait for it runs out. Nothing here faults or hangs the GPU.
"""
import ctypes
import time

import pytest

from tests.test_gpu_shared_attention import Batch

gpu = pytest.mark.gpu


def _lib():
    import speculative_decoding_draft_rmsnorm_gb300 as D
    from speculative_decoding_draft_rmsnorm_gb300 import _build, decode
    D.load()  # the product library (built by the package's build step, with this one)
    if not _build.up_to_date(_build.WAIT_TEST_LIB_PATH):
        _build.build()
    lib = ctypes.CDLL(_build.WAIT_TEST_LIB_PATH)
    decode.declare(lib)
    lib.dflash_last_error.restype = ctypes.c_char_p
    return D, lib


def test_the_hooks_are_in_the_test_library_only():
    D, lib = _lib()
    product = ctypes.CDLL(D.lib_path())
    lib.dflash_test_withhold_norm_row.argtypes = [ctypes.c_longlong]
    for name in ("dflash_test_withhold_prefix_tile", "dflash_test_withhold_norm_row"):
        assert hasattr(lib, name) and not hasattr(product, name)


def _attend(lib, D, b, f32, window, ws, status):
    """The call that Batch.run makes, of the test library."""
    import torch
    n, hq, dh = b.q.shape
    out = torch.zeros(n, hq, dh, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)
    lse = torch.zeros(n, hq, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    rc = lib.dflash_decode_attention_shared(
        p(b.q), hq * dh, p(b.k), p(b.v), p(b.table), b.table.stride(0), p(b.ln), p(b.st), p(b.px), n, b.px.numel(), hq, b.k.shape[2], dh,
        b.k.shape[0], b.k.shape[1], b.table.shape[1], int(b.lens.max()), 0.0, window, D.OUT_F32 if f32 else D.OUT_BF16, p(out), p(lse), p(ws),
        ws.numel(), D.FLAG_FORCE_SHARE, p(status) if status is not None else None, torch.cuda.current_stream().cuda_stream)
    assert rc == 0, lib.dflash_last_error().decode()
    return out, lse


@gpu
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("groups,ps,hq,hkv,dh,window,block,tile", [
    ([(2000, [2100, 2007, 2000, 1999, 0])], 16, 8, 2, 128, 0, 0, 0),               # a tile a block
    ([(2000, [2100, 2007, 2000, 30])], 5, 8, 2, 64, 0, 7, 0),                      # row by row
    ([(900, [901, 1200]), (5000, [5001 + i for i in range(40)])], 16, 40, 8, 128, 0, 60, 3),  # units cut between blocks, parts of many
    ([(700, [700] * 90), (64, [70] * 9)], 16, 16, 2, 64, 500, 3, 0),
])
def test_a_withheld_tile_of_a_prefix(groups, ps, hq, hkv, dh, window, block, tile, f32):
    import torch
    D, lib = _lib()
    b = Batch(groups, ps, hq, hkv, dh, seed=block, before=2, after=1)
    want = b.run(f32, window=window)  # the product's
    shares = torch.zeros(len(b.lens), dtype=torch.bool)
    for g, (p, _) in enumerate(groups):
        for r in range(b.starts[g], b.starts[g + 1]):
            shares[r] = bool(b.lens[r] >= p)
    assert int(shares.sum()) > 1 and not bool(shares.all())
    ws = D.alloc_workspace(D.shared_workspace_size(len(b.lens), len(groups), hq, hkv, dh, int(b.lens.max()), window))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for fill in (0x7f, 0x01):  # what a call may find in a workspace: notes of where parts are that lead far out of it
        for st in (status, None):
            ws.fill_(fill)
            status.zero_()
            assert lib.dflash_test_withhold_prefix_tile(block, tile) == 0
            try:
                torch.cuda.synchronize()
                t0 = time.perf_counter()
                out, lse = _attend(lib, D, b, f32, window, ws, st)
                torch.cuda.synchronize()
                took = time.perf_counter() - t0
            finally:
                assert lib.dflash_test_withhold_prefix_tile(-1, -1) == 0
            assert took < 1.0, f"the timed-out call took {took:.3f} s"
            if st is not None:
                assert status.item() == D.STATUS_TIMEOUT
            # nothing is missing unseen, and what needs no prefix is right
            assert bool(out[shares].isnan().all()) and bool(lse[shares].isnan().all())
            assert torch.equal(out[~shares], want[0][~shares]) and torch.equal(lse[~shares], want[1][~shares])
    status.zero_()
    got = _attend(lib, D, b, f32, window, ws, status)  # the same workspace
    assert status.item() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@gpu
@pytest.mark.parametrize("n,d,f32,residual,group,row", [
    (3000, 4096, False, True, 128, 0),        # 8 warps a row, e4m3 by groups
    (3000, 4096, False, True, 128, 2000),
    (20001, 512, True, False, 0, 7777),       # a warp a row, e4m3 by rows
    (16000, 1024, False, True, None, 15999),  # the last row, its own type
    (1000, 16384, True, False, None, 400),    # a block a row
    (9000, 2560, False, False, 64, 160),
])
def test_a_withheld_row_of_the_norm(n, d, f32, residual, group, row):
    import torch
    D, lib = _lib()
    lib.dflash_test_withhold_norm_row.argtypes = [ctypes.c_longlong]
    gen = torch.Generator(device="cuda").manual_seed(row)
    dt = torch.float32 if f32 else torch.bfloat16
    x = torch.randn(n, d, device="cuda", generator=gen).to(dt)
    r = torch.randn(n, d, device="cuda", generator=gen).to(dt) if residual else None
    w = torch.randn(d, device="cuda", generator=gen)
    eight = group is not None
    kind = D.OUT_E4M3 if eight else D.OUT_F32 if f32 else D.OUT_BF16
    want = D.rms_norm(x, w, residual=r, out_dtype=kind, group_size=group or 0)  # the product's
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = lambda t: None if t is None else t.data_ptr()  # noqa: E731

    def call(st):
        got = [None if t is None else torch.zeros_like(t) for t in want]
        rc = lib.dflash_rms_norm(p(x), d, p(r), d, p(w), p(got[1]), d, p(got[0]), d, p(got[2]), n, d, D.OUT_F32 if f32 else D.OUT_BF16,
                                 D.OUT_F32, kind, group or 0, 1e-6, p(st), torch.cuda.current_stream().cuda_stream)
        assert rc == 0, lib.dflash_last_error().decode()
        return got

    for st in (status, None):
        status.zero_()
        assert lib.dflash_test_withhold_norm_row(row) == 0
        try:
            torch.cuda.synchronize()
            t0 = time.perf_counter()
            got = call(st)
            torch.cuda.synchronize()
            took = time.perf_counter() - t0
        finally:
            assert lib.dflash_test_withhold_norm_row(-1) == 0
        assert took < 1.0, f"the timed-out call took {took:.3f} s"
        assert st is None or status.item() == D.STATUS_TIMEOUT
        # the row and those behind it of the same warps are NaN, every other row is right
        lost = got[0].float().isnan().all(1)
        at = lost.nonzero()[:, 0].tolist()
        step = at[1] - at[0] if len(at) > 1 else n
        assert at == list(range(row, n, step))
        assert step >= torch.cuda.get_device_properties(0).multi_processor_count
        for a, b in zip(got, want):
            if a is not None:
                assert torch.equal(a[~lost].view(torch.uint8), b[~lost].view(torch.uint8))
        if eight:
            assert bool(got[2][lost].isnan().all())
    status.zero_()
    got = call(status)
    assert status.item() == 0
    for a, b in zip(got, want):
        assert (a is None) == (b is None) and (a is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8)))
