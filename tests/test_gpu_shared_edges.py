"""Far ends of a step over a shared prompt: offsets past 32 bits, pages used twice, very many rows, outputs in place.

Tolerances are those of each operator's own tests, by whose checks outputs are compared.
"""
import numpy as np
import pytest

from tests.test_gpu_rms_norm import check as check_norm
from tests.test_gpu_rms_norm import inputs as norm_inputs
from tests.test_gpu_rotary_axes import check as check_axes
from tests.test_gpu_shared_attention import Batch, cu
from tests.test_gpu_shared_prefixes import define as define_prefixes

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


@pytest.mark.parametrize("ps", [16, 10])
def test_pools_past_32_bits(ps):
    # 2^21 rows of 2 KB: elements and bytes of the last pages lie past 2^31 and 2^32
    import torch
    b = Batch([(300, [310, 330, 305]), (150, [150, 151])], ps, 16, 8, 128, seed=1)
    near, pages = b.k.shape[0], 2 ** 21 // ps + 200
    for name in ("k", "v"):
        far = torch.empty(pages, ps, 8, 128, device="cuda", dtype=torch.bfloat16)
        far[-near:] = getattr(b, name)
        setattr(b, name + "_far", far)
    at = b.table + (b.table >= 0).int() * (pages - near)
    status = torch.zeros(1, device="cuda", dtype=torch.int32)
    for flags in (D().FLAG_FORCE_SHARE, 0):
        got = D().decode_attention_shared(b.q, b.k_far, b.v_far, at, b.ln, b.st, b.px, max_ctx_len=330, return_lse=True, flags=flags, status=status)
        b.check(got)
    assert status.item() == 0
    # and k, v of new tokens to the last slots
    n = 5
    x = torch.randn(n, 32, 128, device="cuda").to(torch.bfloat16)
    slot = torch.arange(pages * ps - n, pages * ps, device="cuda", dtype=torch.int32).flip(0)
    pos = torch.arange(3 * n, device="cuda", dtype=torch.int32).view(3, n)
    freq, _ = D().rotary_frequencies(128)
    axes = D().rotary_sections((16, 24, 24))
    D().rotary_axes(x[:, :16], pos, axes, freq, k=x[:, 16:24], k_out=b.k_far, v=x[:, 24:], v_out=b.v_far, slot=slot, status=status)
    check_axes(b.k_far.view(-1, 8, 128)[slot.long()], x[:, 16:24], pos, axes, freq)
    assert torch.equal(b.v_far.view(-1, 8, 128)[slot.long()], x[:, 24:]) and status.item() == 0


def test_rows_of_tables_past_32_bits():
    import torch
    b = Batch([(300, [310, 330, 305])], 16, 8, 2, 64, seed=2)
    step = 2 ** 30 + 8
    wide = torch.empty(2 * step + b.table.shape[1], device="cuda", dtype=torch.int32)
    far = wide.as_strided(b.table.shape, (step, 1))
    far.copy_(b.table)
    px = D().shared_prefixes(far, b.ln, b.st, page_size=16)
    assert px.tolist() == define_prefixes(b.table.cpu().numpy(), b.lens, b.st.tolist(), 16)
    b.table = far
    b.check(b.run())


def test_one_page_again_and_again():
    # every entry of every row is the same page; the prefix is whatever is shared
    import torch
    b = Batch([(16, [16])], 16, 8, 2, 64, seed=3)
    b.lens = np.array([333, 200, 640, 77], np.int32)
    b.table = torch.full((4, 40), int(b.table[0, 0]), device="cuda", dtype=torch.int32)
    b.q = torch.randn(4, 8, 64, device="cuda").to(torch.bfloat16)
    b.ln, b.st = cu(b.lens), cu([0, 4])
    b.px = D().shared_prefixes(b.table, b.ln, b.st, page_size=16)
    assert b.px.tolist() == [77]
    for p in (77, 200, 333):
        b.px.fill_(p)
        b.check(b.run(True))


def test_many_sequences_in_groups_of_two():
    rng = np.random.default_rng(5)
    b = Batch([(64, [int(x) for x in rng.integers(64, 120, 2)]) for _ in range(1030)], 16, 2, 2, 64, seed=4)
    for flags in (4, 0):
        b.check(b.run(flags=flags))
        assert b.status == 0


@pytest.mark.parametrize("f32", [False, True])
def test_norm_of_rows_past_32_bits(f32):
    import torch
    x, r, w = norm_inputs(3, 2560, f32)
    step = 2 ** 31 + 64 if not f32 else 2 ** 30 + 64
    wide = torch.empty(2 * step + 2560, device="cuda", dtype=x.dtype)
    far = wide.as_strided((3, 2560), (step, 1))
    far.copy_(x)
    want = D().rms_norm(x, w, residual=r)
    got = D().rms_norm(far, w, residual=r, residual_out=far)
    assert got[1].data_ptr() == far.data_ptr()
    assert torch.equal(got[0], want[0]) and torch.equal(far, want[1])
    check_norm((got[0], far, None), x, r, w)


@pytest.mark.parametrize("d", [1, 3, 8, 64])
def test_norm_of_very_many_rows(d):
    import torch
    n = 1500001
    x, r, w = norm_inputs(n, d, False, seed=d)
    check_norm(D().rms_norm(x, w, residual=r), x, r, w)
    check_norm(D().rms_norm(x, w, out_dtype=D().OUT_E4M3), x, None, w)


@pytest.mark.parametrize("n,d", [(9000, 2560), (5000, 5003), (4000, 4097)])
@pytest.mark.parametrize("f32", [False, True])
def test_norm_of_many_rows_in_place(n, d, f32):
    import torch
    x, r, w = norm_inputs(n, d, f32)
    want = D().rms_norm(x, w, residual=r)
    x1, r1 = x.clone(), r.clone()
    got = D().rms_norm(x1, w, residual=r1, residual_out=r1, out=x1)
    assert torch.equal(got[0], want[0]) and torch.equal(r1, want[1]) and torch.equal(x1, want[0])
    # two at once on two streams
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = [D().rms_norm(x, w, residual=r, stream=s) for s in (a, b, a, b)]
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], want[0]) and torch.equal(o[1], want[1]) for o in outs)
