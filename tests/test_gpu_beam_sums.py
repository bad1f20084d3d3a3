"""The log-sums of dflash_beam_select over logits of any size, against 64 bits.

A log-sum is off by what its exponentials are: 2 ulp (2^-22) each, and as much again for every change of the maximum that a
term is relative to (a few in a thread, then in the warp, the block and the merge): 2^-19 together. A score adds its
own rounding, 2^-24."""
import numpy as np
import pytest

from tests import decode_ref as R

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def check(got, x, s, k):
    want = R.beams(x.double().cpu().numpy(), s.cpu().numpy(), k)
    assert np.array_equal(got["tokens"].cpu().numpy(), want[1])
    assert np.array_equal(got["parents"].cpu().numpy(), want[2])
    have = got["scores"].double().cpu().numpy()
    assert np.all(np.abs(have - want[0]) <= 2.0 ** -19 + 2.0 ** -24 * np.abs(want[0]))


SIZES = [0.0, 100.0, 200.0, 1000.0, 4000.0, 1e4, 1e5, 1e6, 2.0 ** 24, 3e7, 5e7, 1.2e8, 1e9, 1e30]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("vocab", [1000, 5003, 151936])
def test_log_sums_of_large_logits(vocab, f32):
    import torch
    g = torch.Generator(device="cuda").manual_seed(vocab)
    at = torch.tensor([sign * a for a in SIZES for sign in (1, -1)], device="cuda")
    x = 2.5 * torch.randn(len(at), 2, vocab, device="cuda", generator=g) + at[:, None, None]
    x = x.to(torch.float32 if f32 else torch.bfloat16)
    s = -10 * torch.rand(len(at), 2, device="cuda", generator=g)
    check(D().beam_select(x, s, beams_out=4), x, s, 4)


@pytest.mark.parametrize("f32", [False, True])
def test_beams_of_different_sizes_are_ranked_alike(f32):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    n, vocab = 12, 20011
    at = torch.tensor([[0.0, 300.0, -900.0, 3000.0]], device="cuda")
    x = 2.5 * torch.randn(n, 4, vocab, device="cuda", generator=g) + at[..., None]
    x = x.to(torch.float32 if f32 else torch.bfloat16)
    s = -0.1 * torch.rand(n, 4, device="cuda", generator=g)
    check(D().beam_select(x, s, beams_out=16), x, s, 16)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,w,k,vocab,pad", [
    (6, 3, 8, 32003, 0), (3, 8, 8, 151936, 0), (40, 4, 8, 20000, 1), (75, 4, 4, 20003, 0), (200, 5, 7, 5000, 0), (1, 32, 32, 40001, 3),
    (3, 4, 16, 1001, 0),
])
def test_equal_beams_tie_however_their_rows_lie(n, w, k, vocab, pad, f32):
    """Beams of equal logits and equal scores: the candidates tie in pairs, the lower beam first. Rows of an odd length
    (or stride) are aligned differently, and rows laid end to end are cut at different places."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = torch.empty(n, w, vocab + pad, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16)[:, :, :vocab]
    x.copy_(2.5 * torch.randn(n, 1, vocab, device="cuda", generator=g))
    s = torch.full((n, w), -1.0, device="cuda")
    x[::2, w - 1, ::7] = -float("inf")  # every other request: the last beam is another
    if w > 2:
        x[:, 1] = 2.5 * torch.randn(n, vocab, device="cuda", generator=g)  # and the second
    x[:, :, 3] = 0.0
    x[:, 0, 3] = -0.0
    check(D().beam_select(x, s, beams_out=k), x, s, k)
    s[:, 0] = -float("inf")             # not live: no candidates, whatever its logits
    check(D().beam_select(x, s, beams_out=k), x, s, k)
    s = -1.0 - 0.37 * torch.arange(w, device="cuda").float().repeat(n, 1)
    check(D().beam_select(x, s, beams_out=k), x, s, k)


def test_overlapping_outputs_are_refused():
    import torch
    n, w, vocab = 6, 4, 500
    x = torch.randn(n, w, vocab, device="cuda")
    flat = torch.zeros(4 * n * w, device="cuda")
    s = flat[:n * w].view(n, w)
    ints = torch.zeros(2 * n * w, dtype=torch.int32, device="cuda")
    flags = torch.zeros(2 * n * w, dtype=torch.bool, device="cuda")
    fin = flags[:n * w].view(n, w)

    def refused(**out):
        with pytest.raises(D().DFlashError, match="overlap|alias"):
            D().beam_select(x, s, finished=fin, eos=1, out=out)

    for off in (0, 1, 5, n * w - 1):
        refused(scores=flat[off:off + n * w].view(n, w))
        refused(finished=flags[off:off + n * w].view(n, w))
        refused(tokens=ints[:n * w].view(n, w), parents=ints[off:off + n * w].view(n, w))
        refused(tokens=flat.view(torch.int32)[off:off + n * w].view(n, w))
    want = D().beam_select(x, s, finished=fin, eos=1)
    out = dict(scores=flat[n * w:2 * n * w].view(n, w), tokens=ints[:n * w].view(n, w), parents=ints[n * w:].view(n, w),
               finished=flags[n * w:].view(n, w))
    got = D().beam_select(x, s, finished=fin, eos=1, out=out)
    assert all(torch.equal(got[k], want[k]) for k in want)
