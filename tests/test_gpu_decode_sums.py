"""The sums of dflash_decode_attention_paged over many rows, where an error that is always of one sign adds up."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


@pytest.mark.parametrize("hq", [4, 16])
@pytest.mark.parametrize("f32", [False, True])
def test_sums_of_a_long_range_do_not_drift(hq, f32):
    """Values of 1 and 1 + 2^-7, half of each: a mean lies within 1e-4 of the border between these two bf16 numbers, and
    the output is the one on its side unless it is nearer to the border than the sums are exact.

    There are as many equal sequences as warps, so that one warp adds up all 60000 rows of one. Tolerance, relative: a
    rounded addition of a step to a sum that has grown to i of N steps is off by at most 2^-24 i/N of the result, evenly
    spread, so N = 3750 of them have a standard deviation of 2^-24 sqrt(N) / 3 = 1.2e-6, numerator and weight each; 6
    deviations of their sum are 1.1e-5. Within a step at most 4 additions are cut off at 2^-23, which is 5e-7. Weights:
    16 bits, each off by 2^-17 at most to either side: 2^-17 / sqrt(60000) is nothing. (Sums that are cut off at every
    step are 5e-5 to 1e-4 too small.)"""
    import torch
    rows, dh, ps = 60000, 128, 16
    seqs = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    rng = np.random.default_rng(3)
    k = torch.from_numpy(rng.standard_normal((rows // ps, ps, 1, dh)).astype(np.float32)).to(torch.bfloat16)
    v = torch.from_numpy((1.0 + 2.0 ** -7 * (rng.random((rows // ps, ps, 1, dh)) < 0.5)).astype(np.float32)).to(torch.bfloat16)
    q = torch.from_numpy((0.8 * rng.standard_normal((1, hq, dh))).astype(np.float32)).to(torch.bfloat16)
    table = torch.arange(rows // ps, dtype=torch.int32, device="cuda").repeat(seqs, 1)
    lens = torch.full((seqs,), rows, dtype=torch.int32, device="cuda")
    got = D().decode_attention_paged(q.cuda().expand(seqs, hq, dh), k.cuda(), v.cuda(), table, lens, max_ctx_len=rows,
                                     out_dtype=D().OUT_F32 if f32 else D().OUT_BF16)
    assert bool((got == got[:1]).all())
    s = q[0].double().numpy() @ k.view(rows, dh).double().numpy().T / np.sqrt(dh)
    p = np.exp(s - s.max(-1, keepdims=True))
    want = (p / p.sum(-1, keepdims=True)) @ v.view(rows, dh).double().numpy()
    have, tol = got[0].double().cpu().numpy(), 1.2e-5
    if f32:
        assert np.abs(have - want).max() <= tol * want.max()
        return
    border = 1.0 + 2.0 ** -8
    clear = np.abs(want - border) > tol * border
    assert clear.sum() > clear.size // 4 and (want[clear] < border + 1e-4).all()
    assert np.array_equal(have[clear], np.where(want > border, 1.0 + 2.0 ** -7, 1.0)[clear])


@pytest.mark.parametrize("hq", [1, 8, 16])
def test_weights_keep_24_bits_for_f32_outputs(hq):
    """Two rows, with scores 0 and -t and values 0 and 1: the output is w / (1 + w), w = exp(-t).

    Relative: the exponential 2^-22, its argument (the scale and one FMA) 2 t 2^-24 with t <= 2, the weight 2^-24, the
    sum, its reciprocal and their product 2^-24 each: 2^-21 together. (16 bits of the weight are off by up to 2^-17.)"""
    import torch
    n, dh = 256, 64
    t = torch.arange(1, n + 1).double() / 128  # exact in bf16
    k, v = torch.zeros(n, 16, 1, dh, dtype=torch.bfloat16), torch.full((n, 16, 1, dh), float("nan"), dtype=torch.bfloat16)
    k[:, 1, 0, 0] = -t.to(torch.bfloat16)
    v[:, 0], v[:, 1] = 0.0, 1.0
    q = torch.zeros(n, hq, dh, dtype=torch.bfloat16)
    q[:, :, 0] = 1.0
    table = torch.arange(n, dtype=torch.int32, device="cuda")[:, None].contiguous()
    lens = torch.full((n,), 2, dtype=torch.int32, device="cuda")
    got = D().decode_attention_paged(q.cuda(), k.cuda(), v.cuda(), table, lens, max_ctx_len=16, scale=1.0, out_dtype=D().OUT_F32)
    w = torch.exp(-t)
    want = (w / (1 + w))[:, None, None]
    assert bool(((got.double().cpu() - want).abs() <= 2.0 ** -21 * want).all())
