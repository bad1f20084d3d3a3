"""dflash_beam_select on the GPU against a sort of every candidate in 64 bits.

Tokens, parents and flags are equal. A score carries half an f32 step (2^-24 of it) and the error of the
log of a sum of positive terms: 2^-21 for each exponential (2 ulp and a rounded product of a few units)
and 2^-24 for each addition on a term's way, at most 64 + vocab / 2048 of them.
"""
import numpy as np
import pytest

from tests import decode_ref as R

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def check(got, logits, scores, k, finished=None, eos=-1):
    f = finished.cpu().numpy() if finished is not None else None
    want = R.beams(logits.double().cpu().numpy(), scores.cpu().numpy(), k, f, eos)
    s = got["scores"].double().cpu().numpy()
    assert np.array_equal(got["tokens"].cpu().numpy(), want[1])
    assert np.array_equal(got["parents"].cpu().numpy(), want[2])
    assert np.array_equal(got["finished"].cpu().numpy(), want[3])
    none = want[1] < 0
    assert np.all(s[none] == -np.inf)
    tol = 2.0 ** -24 * np.abs(want[0][~none]) + 2.0 ** -21 + (64 + logits.shape[2] / 2048) * 2.0 ** -24
    assert np.all(np.abs(s[~none] - want[0][~none]) <= tol)


def draw(n, w, vocab, f32, seed=0, spread=2.5):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (spread * torch.randn(n, w, vocab, device="cuda", generator=g)).to(torch.float32 if f32 else torch.bfloat16)
    return x, -10 * torch.rand(n, w, device="cuda", generator=g)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,w,k,vocab", [(1, 1, 1, 1), (1, 4, 4, 151936), (3, 5, 5, 32003), (7, 1, 32, 1000), (2, 32, 32, 4099),
                                         (40, 3, 7, 257), (5, 2, 9, 3), (1, 8, 2, 20001), (300, 2, 2, 64)])
def test_matches_definition(n, w, k, vocab, f32):
    x, s = draw(n, w, vocab, f32, seed=vocab)
    check(D().beam_select(x, s, beams_out=k), x, s, k)


@pytest.mark.parametrize("f32", [False, True])
def test_finished_dead_and_masked(f32):
    import torch
    n, w, k, vocab = 12, 4, 6, 5003
    x, s = draw(n, w, vocab, f32, seed=2)
    fin = torch.rand(n, w, device="cuda") < 0.4
    fin[0], fin[1] = True, False
    inf = float("inf")
    s[2] = -inf                     # no live beam
    s[3, 1:] = -inf                 # the first step of a search: one live beam
    x[4, :, 10:] = -inf             # few tokens left
    x[5] = -inf                     # every token masked
    x[6, 1] = -inf                  # one beam without tokens
    x[7, 2, 77], x[7, 3, 5] = float("nan"), inf  # beams without candidates
    s[8, 0] = float("nan")
    x[9] = torch.finfo(x.dtype).min
    x[9, :, 100:140] = 1.0
    x[10, :, :] = torch.finfo(x.dtype).min  # all equal, at the type's lowest value
    check(D().beam_select(x, s, beams_out=k, finished=fin, eos=9), x, s, k, fin, 9)
    check(D().beam_select(x, s, beams_out=k, eos=9), x, s, k, None, 9)


@pytest.mark.parametrize("f32", [False, True])
def test_ties_go_to_the_lowest_index(f32):
    import torch
    n, w, k, vocab = 6, 3, 8, 40000
    x, _ = draw(n, w, vocab, f32, seed=3)
    x = x.round()                 # few distinct values: many ties inside a beam
    x[0] = 0.0                    # a constant row
    x[1, :] = x[1, :1]            # equal beams with equal scores: ties across beams (rows of one alignment: equal sums)
    x[2, :, ::2], x[2, :, 1::2] = 1.0, 0.0
    x[3] = torch.sort(x[3], dim=-1).values                   # ascending: every batch improves
    x[4] = torch.sort(x[4], dim=-1, descending=True).values
    x[5, :, -8:] = 30.0           # all winners at the end
    s = torch.full((n, w), -1.0, device="cuda")
    check(D().beam_select(x, s, beams_out=k), x, s, k)


def test_strides_and_misaligned_rows():
    import torch
    big = torch.randn(4, 6, 3001, device="cuda").to(torch.bfloat16)
    s = -torch.rand(4, 3, device="cuda")
    for off in range(1, 9):
        x = big[:, ::2, off:off + 2950]
        check(D().beam_select(x, s), x, s, 3)


def test_graph_stream_and_preallocated():
    import torch
    x, s = draw(5, 4, 9000, False, seed=5)
    want = D().beam_select(x, s)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = D().beam_select(x, s, stream=st)
    torch.cuda.synchronize()
    out = {k: torch.empty_like(v) for k, v in want.items()}
    ws = D().alloc_workspace(D().beam_workspace_size(5, 4, 4, 9000))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D().beam_select(x, s, out=out, workspace=ws)
    x.copy_(draw(5, 4, 9000, False, seed=6)[0])
    g.replay()
    again = D().beam_select(x, s)
    for k in want:
        assert torch.equal(got[k], want[k]) and torch.equal(out[k], again[k])


def test_refusals():
    import torch
    d = D()
    x, s = draw(2, 3, 100, False)
    fin = torch.zeros(2, 3, dtype=torch.bool, device="cuda")
    for exc, args, kw in [(TypeError, (x.half(), s), {}), (TypeError, (x, s.double()), {}), (ValueError, (x, s[:1]), {}),
                          (ValueError, (x.transpose(1, 2), s), {}), (TypeError, (x, s), dict(finished=fin.int(), eos=1)),
                          (ValueError, (x, s), dict(beams_out=0)), (d.DFlashError, (x, s), dict(beams_out=33)),
                          (d.DFlashError, (x, s), dict(finished=fin)), (d.DFlashError, (x, s), dict(eos=100)),
                          (d.DFlashError, (x, s), dict(eos=-2)), (ValueError, (x, s.cpu()), {}),
                          (d.DFlashError, (x, s), dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")))]:
        with pytest.raises(exc):
            d.beam_select(*args, **kw)
    with pytest.raises(d.DFlashError):
        d.beam_select(torch.zeros(1, 33, 8, device="cuda"), torch.zeros(1, 33, device="cuda"))
    empty = d.beam_select(x[:0], s[:0])
    assert empty["tokens"].shape == (0, 3)
