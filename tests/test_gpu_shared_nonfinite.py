"""dflash_decode_attention_shared where seen rows or queries hold NaN or infinities: as dflash_decode_attention_paged, shared or not.

By the definition a NaN score makes the weights' sum NaN, and with it the output and the log-sum; a log-sum of -inf means that there
is no weight at all.
"""
import numpy as np
import pytest

from tests.test_gpu_shared_attention import Batch, D

pytestmark = pytest.mark.gpu
PREFIX = 600


def _batch(ps=16, dh=128):
    # groups that share, in which some sequences do not; a sequence in no group
    return Batch([(PREFIX, [610, 605, 700, 300, 600]), (200, [205, 230, 0])], ps, 8, 2, dh, seed=40, before=1)


def _row(b, r, j):
    ps = b.k.shape[1]
    return b.table[r, j // ps].item(), j % ps


def _calls(b, f32, window=0):
    """The paged call's (out, lse), and the shared call's with and without sharing asked for."""
    dtype = D().OUT_F32 if f32 else D().OUT_BF16
    paged = D().decode_attention_paged(*b.args()[:5], max_ctx_len=int(b.lens.max()), window=window, out_dtype=dtype, return_lse=True)
    return paged, [b.run(f32, window=window, flags=flags) for flags in (0, D().FLAG_FORCE_SHARE)]


def _same_kind(paged, got):
    for x, y in zip(paged, got):
        assert bool((x.isnan() == y.isnan()).all())
        assert bool((x.isinf() == y.isinf()).all())
        assert bool((x[x.isinf()] == y[y.isinf()]).all())


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("ps,dh", [(16, 128), (5, 64)])
@pytest.mark.parametrize("row,seen_by", [(0, [1, 2, 3, 4, 5]), (250, [1, 2, 3, 4, 5]), (301, [1, 2, 3, 5]), (599, [1, 2, 3, 5])])
def test_nan_in_a_shared_key(row, seen_by, ps, dh, f32):
    b = _batch(ps, dh)
    for r in seen_by:  # in every page that holds the row (the fourth sequence has its own)
        page, off = _row(b, r, row)
        b.k[page, off, 1, 3] = float("nan")
    paged, got = _calls(b, f32)
    want = np.zeros((len(b.lens), 8), bool)
    want[seen_by, 4:] = True  # the heads of kv head 1
    for out, lse in (paged, *got):
        assert np.array_equal(lse.isnan().cpu().numpy(), want)
        assert np.array_equal(out.isnan().any(-1).cpu().numpy(), want) and np.array_equal(out.isnan().all(-1).cpu().numpy(), want)
    for x in got:
        _same_kind(paged, x)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("window", [0, 50])
def test_nan_in_an_own_key_and_in_a_query(window, f32):
    b = _batch()
    page, off = _row(b, 3, 690)  # of the third sequence's own rows
    b.k[page, off, 0, 0] = float("nan")
    b.q[0, 7, 5] = b.q[2, 6, 100] = b.q[4, 1, 0] = b.q[8, 2, 2] = float("nan")  # ungrouped, sharing, not sharing, without rows
    paged, got = _calls(b, f32, window)
    want = np.zeros((len(b.lens), 8), bool)
    want[3, :4] = want[0, 7] = want[2, 6] = want[4, 1] = True
    for out, lse in (paged, *got):
        assert np.array_equal(lse.isnan().cpu().numpy(), want)
        assert np.array_equal(out.isnan().all(-1).cpu().numpy(), want)
        assert bool((lse[8] == -float("inf")).all()) and bool((out[8] == 0).all())
    for x in got:
        _same_kind(paged, x)


@pytest.mark.parametrize("f32", [False, True])
def test_scores_of_minus_infinity(f32):
    # every score of a head is -inf: no weight, so the log-sum is -inf and the output 0 / 0; some are: they weigh nothing
    import torch
    b = _batch()
    b.q.copy_(b.q.abs())
    live = ~torch.isnan(b.k[..., 0, 0].float())
    own = b.k.clone()
    b.k[:, :, 0][live] = -float("inf")
    paged, got = _calls(b, f32)
    for out, lse in (paged, *got):
        assert bool((lse[:8, :4] == -float("inf")).all()) and bool(out[:8, :4].isnan().all())
        assert bool(lse[:8, 4:].isfinite().all()) and bool(out[:8, 4:].isfinite().all())
    b.k.copy_(own)
    for j in range(PREFIX):
        page, off = _row(b, 1, j)
        b.k[page, off, 0] = -float("inf")
    b.lens[5] = 599  # of the prefix alone: it has no other row
    b.ln[5] = 599
    paged, got = _calls(b, f32)
    for out, lse in (paged, *got):
        assert bool(lse[1:4].isfinite().all()) and bool(out[1:4].isfinite().all())
    for x in got:
        _same_kind(paged, x)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_finite(bad, f32):
    # a weight is added in terms, p = h + r with r of either sign or 0: h inf + r inf is inf or NaN. No other column sees it
    b = _batch()
    for r, j in ((1, 77), (3, 650)):
        page, off = _row(b, r, j)
        b.v[page, off, 0, 9] = bad
    paged, got = _calls(b, f32)
    for out, lse in (paged, *got):
        hit = out[[1, 2, 3, 5], :4, 9]
        assert bool((hit.isnan() | (hit == bad)).all())
        rest = out.clone()
        rest[[1, 2, 3, 5], :4, 9] = 0
        assert bool(rest.isfinite().all()) and bool(lse[:8].isfinite().all())
