"""dflash_decode_attention_paged on the GPU against the definition in 64 bits.

Tolerance of an output, with A = sum p |v| (weights normalised) and ds the error of a score: a score is
a sum of Dh exact products, each addition off by 2^-23 of the absolute sum at most; weights then by 2 ds
relative, the exponential by 2^-21, a weight kept in 16 bits by 2^-16 (24 for an f32 output: 2^-23), and a
running sum of n rows takes n / 16 additions of 16 terms, each off by 2 x 2^-23, before a join of a few
hundred parts. A bf16 output adds half a step, 2^-8 of its value.
"""
import numpy as np
import pytest

from tests import decode_ref as R

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def store(lens, ps, hkv, dh, seed=0, slack=3, share=False):
    """Pools with NaN in every row that no sequence holds, a shuffled table, both with spare room."""
    import torch
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, np.int32)
    per = -(-lens // ps)
    pages = int(per.sum()) + slack
    width = int(per.max(initial=0)) + 2
    table = np.full((len(lens), width), -1, np.int32)
    ids = rng.permutation(pages)
    at = 0
    for r, n in enumerate(per):
        table[r, :n] = ids[at:at + n]
        at += n
    live = np.zeros((pages, ps), bool)
    if share and len(lens) > 1:  # sequence 1 continues sequence 0's pages
        n = min(per[0], per[1])
        table[1, :n] = table[0, :n]
    for r in range(len(lens)):
        j = np.arange(lens[r])
        live[table[r, j // ps], j % ps] = True
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn(pages, ps, hkv, dh, device="cuda", generator=g).to(torch.bfloat16)
    v = torch.randn(pages, ps, hkv, dh, device="cuda", generator=g).to(torch.bfloat16)
    dead = torch.from_numpy(~live).cuda()
    k[dead], v[dead] = float("nan"), float("nan")
    return k, v, torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()


def check(out, lse, q, k, v, table, lens, window=0, scale=0.0, rows=None):
    import torch
    rows = range(len(lens)) if rows is None else rows
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    ln = lens.cpu().numpy()
    want, wl, mass, ds = R.decode(f(q), f(k), f(v), table.cpu().numpy(), ln, window, scale)
    n = np.minimum(ln, window) if window else ln
    rel = 2 * ds[..., None] + 2.0 ** -21 + (n[:, None, None] / 8 + 512) * 2.0 ** -23
    rel = rel + (2.0 ** -16 if out.dtype == torch.bfloat16 else 2.0 ** -23)
    tol = rel * mass + (2.0 ** -8 * np.abs(want) if out.dtype == torch.bfloat16 else 0.0)
    got, gl = f(out), f(lse)
    for r in rows:
        assert np.all(np.abs(got[r] - want[r]) <= tol[r]), r
        if ln[r]:
            lt = ds[r] + 2.0 ** -21 + n[r] * 2.0 ** -24 + 2.0 ** -22 * np.abs(wl[r])
            assert np.all(np.abs(gl[r] - wl[r]) <= lt), r
        else:
            assert np.all(gl[r] == -np.inf) and np.all(got[r] == 0)


def attend(q, k, v, table, lens, longest=None, f32=False, **kw):
    longest = int(lens.max()) if longest is None else longest
    return D().decode_attention_paged(q, k, v, table, lens, max_ctx_len=longest, return_lse=True,
                                      out_dtype=D().OUT_F32 if f32 else D().OUT_BF16, **kw)


def queries(n, hq, dh, seed=1):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (1.5 * torch.randn(n, hq, dh, device="cuda", generator=g)).to(torch.bfloat16)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("lens,ps,hq,hkv,dh", [
    ([1], 16, 1, 1, 64), ([17], 16, 16, 8, 128), ([0, 5, 0, 300, 0], 16, 8, 2, 128), ([64, 65, 63, 1, 16, 15], 16, 12, 2, 64),
    ([2000, 3, 900], 24, 6, 1, 128), ([700] * 9, 5, 16, 1, 128), ([4097], 128, 40, 2, 64), ([33, 31], 1, 7, 7, 128),
    ([100, 2000], 64, 20, 1, 128), ([50] * 300, 16, 4, 4, 64),
])
def test_matches_definition(lens, ps, hq, hkv, dh, f32):
    q = queries(len(lens), hq, dh)
    k, v, table, ln = store(lens, ps, hkv, dh)
    out, lse = attend(q, k, v, table, ln, f32=f32)
    check(out, lse, q, k, v, table, ln)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 4096])
def test_window(window):
    lens = [1, 2, 15, 16, 17, 99, 100, 101, 777]
    q = queries(len(lens), 8, 128)
    k, v, table, ln = store(lens, 16, 2, 128, seed=2)
    # rows before the window may hold anything
    import torch
    kk, vv = k.clone(), v.clone()
    for r, n in enumerate(lens):
        for j in range(0, max(0, n - window)):
            kk[table[r, j // 16], j % 16] = float("nan")
            vv[table[r, j // 16], j % 16] = float("inf")
    out, lse = attend(q, kk, vv, table, ln, f32=True, window=window)
    check(out, lse, q, k, v, table, ln, window)
    torch.cuda.synchronize()


def test_many_ragged_sequences_bounds_and_workers():
    # more sequences than scan chunks, zero-length runs, a bound far above the lengths
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 90, 700)
    lens[rng.random(700) < 0.4] = 0
    q = queries(700, 4, 64)
    k, v, table, ln = store(lens, 16, 2, 64, seed=5)
    import torch
    wide = torch.full((700, 4000), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    out, lse = attend(q, k, v, wide, ln, longest=64000)
    check(out, lse, q, k, v, table, ln)
    out2, lse2 = attend(q, k, v, table, ln)  # another worker count: the same rows, joined elsewhere
    check(out2, lse2, q, k, v, table, ln)


def test_extreme_scores_and_repeated_maxima():
    # scores that grow along the sequence (every step rescales), one huge score, equal scores
    import torch
    lens = [500, 500, 500]
    q = queries(3, 4, 128)
    k, v, table, ln = store(lens, 16, 1, 128, seed=6)
    for r, f in [(0, lambda j: j / 40.0), (1, lambda j: 30.0 if j == 250 else 0.01), (2, lambda j: 0.0)]:
        for j in range(500):
            k[table[r, j // 16], j % 16, 0] = (q[r, 0].float() * (f(j) / 20)).to(torch.bfloat16)
    out, lse = attend(q, k, v, table, ln, f32=True)
    check(out, lse, q, k, v, table, ln)


def test_shared_pages_strided_queries_and_tables():
    import torch
    lens = [300, 300, 40]
    k, v, table, ln = store(lens, 16, 2, 128, seed=7, share=True)
    fused = queries(3, 8 + 4, 128)
    q = fused[:, :8]
    big = torch.full((3, 64), -1, dtype=torch.int32, device="cuda")
    big[:, 8:8 + table.shape[1]] = table
    strided = big[:, 8:8 + table.shape[1]]
    out, lse = attend(q, k, v, strided, ln)
    check(out, lse, q, k, v, table, ln)
    plain, _ = attend(q.contiguous(), k, v, table, ln)
    assert torch.equal(plain, out)


def test_bad_metadata_is_reported_and_the_others_are_computed():
    import torch
    lens = [100, 50, 70, 90]
    q = queries(4, 8, 64)
    k, v, table, ln = store(lens, 16, 2, 64, seed=8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    attend(q, k, v, table, ln, status=status)
    assert status.item() == 0
    bad = ln.clone()
    bad[1], bad[2] = -4, 101
    out, lse = attend(q, k, v, table, bad, longest=100, status=status)
    assert status.item() == D().STATUS_METADATA
    bad[1] = bad[2] = 0  # both count as empty
    check(out, lse, q, k, v, table, bad)
    t2 = table.clone()
    t2[3, 1] = k.shape[0] + 7
    status.zero_()
    out, lse = attend(q, k, v, t2, ln, status=status)
    assert status.item() == D().STATUS_METADATA
    check(out, lse, q, k, v, table, ln, rows=[0, 1, 2])


def test_graph_replays_with_other_lengths_and_two_graphs_share_a_workspace():
    import torch
    lens = [900, 20, 333, 0]
    q = queries(4, 16, 128)
    k, v, table, ln = store(lens, 16, 4, 128, seed=9)
    k = torch.nan_to_num(k)
    v = torch.nan_to_num(v)
    ws = D().alloc_workspace(D().decode_workspace_size(4, 16, 4, 128, 900))
    out = [torch.empty(4, 16, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    lse = [torch.empty(4, 16, device="cuda") for _ in range(2)]
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            D().decode_attention_paged(q, k, v, table, ln, max_ctx_len=900, out=out[i], lse=lse[i], workspace=ws)
        graphs.append(g)
    for now in (lens, [899, 0, 1, 2], [16, 17, 300, 0]):
        now[3] = 0
        ln.copy_(torch.tensor(now, dtype=torch.int32))
        want, wl = attend(q, k, v, table, ln, longest=900)
        for i, g in enumerate(graphs):
            out[i].fill_(3.0)
            g.replay()
            assert torch.equal(out[i], want) and torch.equal(lse[i], wl)


def test_repeatable_and_on_another_stream():
    import torch
    lens = list(range(1, 1500, 97))
    q = queries(len(lens), 32, 128)
    k, v, table, ln = store(lens, 16, 8, 128, seed=10)
    a = attend(q, k, v, table, ln)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b = [attend(q, k, v, table, ln, stream=s) for _ in range(3)]
    torch.cuda.synchronize()
    for x in b:
        assert torch.equal(x[0], a[0]) and torch.equal(x[1], a[1])


def test_a_long_sequence_past_32_bit_offsets():
    # the pools hold 2^32 bytes and more: the last pages lie behind 32-bit byte offsets
    import torch
    hkv, dh, ps = 8, 128, 16
    pages = (1 << 31) // (ps * hkv * dh) + 40  # > 2^31 elements
    k = torch.zeros(pages, ps, hkv, dh, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros_like(k)
    lens = [500, 70]
    sk, sv, st, ln = store(lens, ps, hkv, dh, seed=11, slack=0)
    n = sk.shape[0]
    k[pages - n:], v[pages - n:] = torch.nan_to_num(sk), torch.nan_to_num(sv)
    table = torch.where(st >= 0, st + (pages - n), st)
    q = queries(2, 32, dh)
    out, lse = attend(q, k, v, table, ln)
    small, sl = attend(q, sk, sv, st, ln)
    assert torch.equal(out, small) and torch.equal(lse, sl)
    check(out, lse, q, sk, sv, st, ln)


def test_refusals():
    import torch
    d = D()
    q = queries(2, 8, 64)
    k, v, table, ln = store([20, 30], 16, 2, 64)

    def refused(exc, *args, **kw):
        kw = {**dict(max_ctx_len=30), **kw}
        with pytest.raises(exc):
            d.decode_attention_paged(*args, **kw)

    refused(TypeError, q.float(), k, v, table, ln)
    refused(TypeError, q, k, v.float(), table, ln)
    refused(TypeError, q, k, v, table.long(), ln)
    refused(ValueError, q, k, v[:-1], table, ln)
    refused(ValueError, q, k, v, table[:1], ln)
    refused(ValueError, q, k[:, :, :, :32], v, table, ln)
    refused(ValueError, q, k.transpose(1, 2), v, table, ln)
    refused(ValueError, q.cpu(), k, v, table, ln)
    refused(ValueError, q, k, v, table, ln.cpu())
    refused(ValueError, queries(2, 64, 8).transpose(1, 2), k, v, table, ln)  # heads not contiguous
    refused(d.DFlashError, queries(2, 7, 64), k, v, table, ln)  # 7 heads over 2
    refused(d.DFlashError, q, k, v, table, ln, max_ctx_len=16 * table.shape[1] + 1)
    refused(d.DFlashError, q, k, v, table, ln, window=-1)
    refused(d.DFlashError, q, k, v, table, ln, scale=float("nan"))
    refused(d.DFlashError, q, k, v, table, ln, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    refused(d.DFlashError, queries(2, 8, 96), torch.zeros(4, 16, 2, 96, device="cuda", dtype=torch.bfloat16),
            torch.zeros(4, 16, 2, 96, device="cuda", dtype=torch.bfloat16), table, ln)
    out, lse = attend(q[:0], k, v, table[:0], ln[:0], longest=0)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    out, lse = attend(q, k[:0], v[:0], table[:, :0], torch.zeros_like(ln), longest=0)
    assert torch.equal(out, torch.zeros_like(out)) and bool((lse == -float("inf")).all())
