"""dflash_decode_attention_shared on the GPU against the definition in 64 bits.

Tolerance of an output, with A = sum p |v| (weights normalised) and ds the error of a score: as for a call without shared
rows, a score is a sum of Dh exact products, each addition off by 2^-23 of the absolute sum at most; weights then by
2 ds relative, the exponential by 2^-21, a weight kept in 16 bits by 2^-16 (24 for an f32 output: 2^-23). Sums: 128 rows of a
prefix are 24 additions of the matrix unit at most, each off by 2^-22, and n / 128 such sums are added with two roundings each;
own rows take n / 16 additions of 16 terms, each off by 2^-22; parts are a few hundred: n / 8 + 560 times 2^-23. A bf16
output adds half a step, 2^-8 of its value.
"""
import numpy as np
import pytest

from tests import decode_ref as R

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def cu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Batch:
    """groups: (prefix, lengths) each. The sequences that are at least `prefix` long hold its rows in the same
    pages; every other row has a page of its own. Rows that nobody holds are NaN."""

    def __init__(self, groups, ps, hq, hkv, dh, seed=0, before=0, after=0, spread=1.0):
        import torch
        rng = np.random.default_rng(seed)
        lens = [7] * before + [n for _, ls in groups for n in ls] + [9] * after
        self.lens = np.array(lens, np.int32)
        starts = before + np.concatenate(([0], np.cumsum([len(ls) for _, ls in groups])))
        self.starts, self.prefix = starts.astype(np.int32), np.array([p for p, _ in groups], np.int32)
        width = max(1, -(-max(lens + [1]) // ps)) + 1
        table, pages = np.full((len(lens), width), -1, np.int32), 0
        live = []
        shared = {}
        for g, (p, _) in enumerate(groups):
            for r in range(starts[g], starts[g + 1]):
                if p and lens[r] >= p:
                    if g not in shared:
                        shared[g] = np.arange(pages, pages + -(-p // ps))
                        pages += len(shared[g])
                    table[r, :len(shared[g])] = shared[g]
        for r, n in enumerate(lens):
            for c in range(-(-n // ps)):
                if table[r, c] < 0:
                    table[r, c] = pages
                    pages += 1
        pages += 3
        ids = rng.permutation(pages).astype(np.int32)
        table = np.where(table >= 0, ids[table], -1).astype(np.int32)
        live = np.zeros((pages, ps), bool)
        for r, n in enumerate(lens):
            j = np.arange(n)
            live[table[r, j // ps], j % ps] = True
        gen = torch.Generator(device="cuda").manual_seed(seed)
        k = torch.randn(pages, ps, hkv, dh, device="cuda", generator=gen).to(torch.bfloat16)
        v = torch.randn(pages, ps, hkv, dh, device="cuda", generator=gen).to(torch.bfloat16)
        dead = torch.from_numpy(~live).cuda()
        k[dead], v[dead] = float("nan"), float("nan")
        q = (1.5 * spread * torch.randn(len(lens), hq, dh, device="cuda", generator=gen)).to(torch.bfloat16)
        self.q, self.k, self.v, self.table = q, k, v, cu(table)
        self.ln, self.st, self.px = cu(self.lens), cu(self.starts), cu(self.prefix)

    def args(self):
        return self.q, self.k, self.v, self.table, self.ln, self.st, self.px

    def run(self, f32=False, longest=None, flags=4, **kw):
        import torch
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = D().decode_attention_shared(*self.args(), max_ctx_len=int(self.lens.max(initial=0)) if longest is None else longest, return_lse=True,
                                          out_dtype=D().OUT_F32 if f32 else D().OUT_BF16, status=status, flags=flags, **kw)
        self.status = status.item()
        return got

    def check(self, got, window=0, scale=0.0, rows=None):
        check(got, self, window, scale, rows)


def check(got, b, window=0, scale=0.0, rows=None):
    import torch
    out, lse = got
    f = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, wl, mass, ds = R.decode(f(b.q), f(b.k), f(b.v), b.table.cpu().numpy(), b.lens, window, scale)
    n = np.minimum(b.lens, window) if window else b.lens
    rel = 2 * ds[..., None] + 2.0 ** -21 + (n[:, None, None] / 8 + 560) * 2.0 ** -23
    rel = rel + (2.0 ** -16 if out.dtype == torch.bfloat16 else 2.0 ** -23)
    tol = rel * mass + (2.0 ** -8 * np.abs(want) if out.dtype == torch.bfloat16 else 0.0)
    o, l = f(out), f(lse)
    for r in range(len(b.lens)) if rows is None else rows:
        assert np.all(np.abs(o[r] - want[r]) <= tol[r]), (r, np.abs(o[r] - want[r]).max())
        if b.lens[r]:
            lt = ds[r] + 2.0 ** -21 + n[r] * 2.0 ** -24 + 2.0 ** -22 * np.abs(wl[r])
            assert np.all(np.abs(l[r] - wl[r]) <= lt), (r, np.abs(l[r] - wl[r]).max())
        else:
            assert np.all(l[r] == -np.inf) and np.all(o[r] == 0)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("groups,ps,hq,hkv,dh", [
    ([(0, [1])], 16, 1, 1, 64),
    ([(128, [130, 129])], 16, 1, 1, 64),
    ([(128, [128, 128])], 16, 2, 1, 128),                                      # nothing of their own
    ([(700, [720, 711, 703, 719])], 16, 16, 8, 128),
    ([(129, [140] * 5), (1000, [1001, 1300]), (0, [5, 6]), (255, [256])], 16, 8, 2, 128),
    ([(257, [300] * 33)], 24, 12, 2, 64),
    ([(640, [650 + i for i in range(40)])], 5, 16, 1, 128),                    # 640 rows of the product
    ([(300, [301] * 9), (200, [233] * 70)], 64, 40, 8, 128),
    ([(2000, [2100] * 3)], 1, 7, 7, 128),
    ([(513, [600, 514])], 128, 272, 2, 64),                                    # groups of 136 heads
    ([(160, [170 + i % 7 for i in range(4)]) for _ in range(60)], 16, 4, 4, 64),
    ([(5000, [5001, 5050, 5100])], 16, 20, 4, 128),
])
def test_matches_definition(groups, ps, hq, hkv, dh, f32):
    b = Batch(groups, ps, hq, hkv, dh, seed=len(groups))
    for flags in (D().FLAG_FORCE_SHARE, 0):
        b.check(b.run(f32, flags=flags))
        assert b.status == 0


@pytest.mark.parametrize("prefix", [1, 2, 15, 16, 17, 63, 64, 65, 100, 127, 128, 129, 143, 144, 255, 256, 257, 384, 500])
@pytest.mark.parametrize("dh", [64, 128])
def test_every_end_of_a_prefix(prefix, dh):
    b = Batch([(prefix, [prefix + 3, prefix, prefix + 40])], 16, 8, 2, dh, seed=prefix)
    b.check(b.run(True))
    b.check(b.run(False))


@pytest.mark.parametrize("f32", [False, True])
def test_short_empty_and_ungrouped_sequences(f32):
    # the first sequences are no part of the prefix; some have no rows; some are in no group
    b = Batch([(300, [10, 0, 305, 299, 400, 0]), (0, []), (200, [0, 0]), (150, [149, 3]), (600, [700])], 16, 8, 2, 128, seed=5, before=3, after=2)
    b.check(b.run(f32))
    b.check(b.run(f32, longest=5 * 16 * 9))
    assert b.status == 0


@pytest.mark.parametrize("window", [1, 16, 100, 129, 300, 1000, 4096])
@pytest.mark.parametrize("f32", [False, True])
def test_window(window, f32):
    import torch
    groups = [(900, [900, 905, 1200, 950]), (400, [401, 430, 0, 390]), (1500, [1501 + 7 * i for i in range(20)])]
    b = Batch(groups, 16, 8, 2, 128, seed=window)
    k, v, table = b.k.clone(), b.v.clone(), b.table.clone()
    # rows that no window reaches may hold anything, and their pages may be gone
    seen = torch.zeros(b.k.shape[:2], dtype=torch.bool)
    for r, n in enumerate(b.lens):
        j = torch.arange(max(0, n - window), n)
        seen[b.table[r].cpu()[j // 16].long(), j % 16] = True
        table[r, :max(0, n - window) // 16] = -7
    b.k[~seen.cuda()], b.v[~seen.cuda()] = float("nan"), float("inf")
    keep, b.table = b.table, table
    got = b.run(f32, window=window)
    assert b.status == 0
    b.k, b.v, b.table = k, v, keep
    b.check(got, window)


@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_scale_and_peaked_scores(scale):
    b = Batch([(1000, [1010] * 12)], 16, 8, 2, 128, seed=7, spread=3.0)
    b.check(b.run(True, scale=scale), scale=scale)
    b.check(b.run(False, scale=scale), scale=scale)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("at", [0, 5, 16, 100, 127, 128, 140, 300, 999])
def test_scores_that_leap(at, f32):
    # one key far above all others, in some heads' eyes only: what came before weighs nothing, whatever tile it came in
    import torch
    b = Batch([(1000, [1001, 1005, 1003, 1009])], 16, 8, 2, 128, seed=at)
    page, off = b.table[0, at // 16].item(), at % 16
    q = b.q.view(4, 2, 4, 128)
    b.k[page, off, 0] = (q[1, 0, 2].float() * 20).to(torch.bfloat16)
    b.k[page, off, 1] = (q[3, 1, 0].float() * 5).to(torch.bfloat16)
    b.check(b.run(f32))


def test_masked_keys_hold_anything():
    # keys of the last tile that lie behind the prefix are NaN (Batch) and inf here
    import torch
    b = Batch([(200, [200, 200, 200])], 16, 4, 1, 128, seed=8)
    want = b.run(True)
    bad = torch.isnan(b.k.float())
    b.k[bad], b.v[bad] = float("inf"), float("-inf")
    got = b.run(True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("window", [1, 20, 128, 300, 400, 611, 1000])
@pytest.mark.parametrize("ps", [5, 16])
def test_rows_that_other_windows_see_hold_anything(window, ps):
    # lengths 600 to 1400 on 600 shared rows: what the longest do not see is inf or NaN to them, in K and V
    import torch
    b = Batch([(600, [600, 601, 617, 650, 700, 790, 899, 900, 901, 1100, 1199, 1200, 1400])], ps, 16, 2, 64, seed=window)
    b.check(b.run(True, window=window), window=window)
    assert b.status == 0
    want = b.run(window=window)
    for r in (3, 6, 11, 12):
        end = b.lens[r] - window  # rows before it are outside the windows of r and of all behind it
        if end <= 0:
            continue
        keep = b.k.clone(), b.v.clone()
        j = torch.arange(end, device="cuda")
        pages, rows = b.table[r, (j // ps).long()].long(), (j % ps).long()
        for bad in (float("nan"), float("inf")):
            b.k[pages, rows], b.v[pages, rows] = bad, -bad
            got = b.run(window=window)
            assert all(torch.equal(x[r:], y[r:]) for x, y in zip(got, want))
        b.k, b.v = keep


@pytest.mark.parametrize("window", [0, 300])
def test_more_groups_than_a_block_of_threads(window):
    rng = np.random.default_rng(3)
    groups = [(int(rng.integers(50, 200)), [200 + int(x) for x in rng.integers(0, 160, rng.integers(0, 3))]) for _ in range(1500)]
    b = Batch(groups, 16, 2, 1, 64, seed=21, before=3, after=2)
    b.check(b.run(True, window=window), window=window)
    assert b.status == 0


def test_any_shorter_prefix_gives_the_result():
    import torch
    b = Batch([(1000, [1001, 1040, 1500])], 16, 16, 4, 128, seed=9)
    for p in (0, 1, 130, 512, 999, 1000):
        b.px.fill_(p)
        b.check(b.run(True))
    want = b.run()
    for _ in range(3):  # and the same one the same bits
        got = b.run()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("starts,prefix", [([0, 4, 2, 8], [300, 300, 300]), ([-1, 4, 8], [300, 300]), ([0, 4, 9], [300, 300]), ([0, 4, 8], [-1, 401]),
                                           ([4, 0], [300]), ([0, 8], [1 << 30])])
def test_bad_groups_are_reported_and_share_nothing(starts, prefix):
    b = Batch([(300, [400, 320, 310, 330]), (300, [400, 320, 310, 300])], 16, 8, 2, 64, seed=10)
    b.st, b.px = cu(starts), cu(prefix)
    for flags in (D().FLAG_FORCE_SHARE, 0):
        b.check(b.run(True, flags=flags))
        assert b.status == D().STATUS_METADATA


def test_bad_pages_and_lengths_are_reported():
    import torch
    b = Batch([(300, [310, 320, 330])], 16, 8, 2, 64, seed=11)
    b.k.nan_to_num_(0.0), b.v.nan_to_num_(0.0)
    keep = b.table.clone()
    for bad in (1 << 20, -1):
        b.table = keep.clone()
        b.table[0, 3] = bad  # within the prefix: page 0 is read in its place
        got = b.run(True)
        assert b.status == D().STATUS_METADATA
        b.table[:, 3] = 0
        b.check(got, rows=[0])  # whose pages they are
    b.table = keep
    b.ln = cu([310, 5000, -2])
    got = b.run(True, longest=330)
    assert b.status == D().STATUS_METADATA
    b.lens = np.array([310, 0, 0], np.int32)
    b.check(got)


def test_strided_queries_and_tables():
    import torch
    b = Batch([(260, [300, 290, 270])], 16, 8, 2, 128, seed=12)
    want = b.run(True)
    wide = torch.zeros(3, 20, 128, device="cuda", dtype=torch.bfloat16)
    wide[:, 5:13] = b.q
    table = torch.full((3, b.table.shape[1] + 5), -3, device="cuda", dtype=torch.int32)
    table[:, 2:2 + b.table.shape[1]] = b.table
    b.q, b.table = wide[:, 5:13], table[:, 2:2 + b.table.shape[1]]
    got = b.run(True)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    b.q = b.q[:1].expand(3, 8, 128)
    b.check(b.run(True))


def test_one_graph_follows_lengths_prefixes_and_tables():
    import torch
    a, b = (Batch([(p, [p + 3, p + 90, p + 30]), (2 * p, [2 * p + 1] * 4)], 16, 8, 2, 128, seed=p) for p in (400, 700))
    assert a.k.shape[0] <= b.k.shape[0]
    width, pages = b.table.shape[1], b.k.shape[0]
    table = torch.full((7, width), -1, dtype=torch.int32, device="cuda")
    k, v = torch.zeros_like(b.k), torch.zeros_like(b.v)
    q, ln, px = b.q.clone(), b.ln.clone(), b.px.clone()
    ws = D().alloc_workspace(D().shared_workspace_size(7, 2, 8, 2, 128, 2000))
    out, lse = torch.empty_like(q), torch.empty(7, 8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D().decode_attention_shared(q, k, v, table, ln, b.st, px, max_ctx_len=1401, out=out, lse=lse, workspace=ws,
                                    flags=D().FLAG_FORCE_SHARE)
    for x in (a, b, a):
        table.fill_(-1)
        table[:, :x.table.shape[1]] = x.table
        k[:x.k.shape[0]], v[:x.v.shape[0]] = x.k, x.v
        q.copy_(x.q), ln.copy_(x.ln), px.copy_(x.px)
        g.replay()
        x.check((out, lse))
    assert out._version >= 1 and lse._version >= 1


def test_two_calls_at_once():
    import torch
    sets = [Batch([(2000 + 500 * i, [2600, 2700, 2800] * 3), (100, [900] * 5)], 16, 32, 4, 128, seed=30 + i) for i in range(2)]
    want = [s.run() for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        got = []
        for s, st in zip(sets, streams):
            got.append(D().decode_attention_shared(*s.args(), max_ctx_len=2800, return_lse=True, stream=st, flags=4))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


@pytest.mark.parametrize("hq,hkv", [(16, 8), (32, 8), (40, 1), (272, 2)])
@pytest.mark.parametrize("window", [0, 100])
def test_workspaces_grow_with_the_call(hq, hkv, window):
    size = D().shared_workspace_size
    for longest in (0, 1, 16, 500, 40000):
        for groups in (0, 1, 50):
            sizes = [size(n, groups, hq, hkv, 128, longest, window) for n in range(1, 400)]
            assert sizes == sorted(sizes), longest
    for n in (1, 7, 150, 1000):
        sizes = [size(n, 3, hq, hkv, 128, c, window) for c in range(0, 3000, 7)]
        assert sizes == sorted(sizes), n
        sizes = [size(n, g, hq, hkv, 128, 900, window) for g in range(0, 1000)]
        assert sizes == sorted(sizes), n


def test_a_smaller_batch_in_the_largest_ones_workspace():
    import torch
    b = Batch([(600, [700 + i for i in range(30)])] * 2, 16, 8, 2, 128, seed=13)
    ws = D().alloc_workspace(D().shared_workspace_size(60, 2, 8, 2, 128, 1000))
    ws.fill_(0xff)
    b.check(b.run(True, workspace=ws))
    for m in (30, 7, 1):
        out, lse = D().decode_attention_shared(b.q[:m], b.k, b.v, b.table[:m], b.ln[:m], cu([0, m]), b.px[:1], max_ctx_len=729, return_lse=True,
                                               workspace=ws, out_dtype=D().OUT_F32, flags=4)
        s = Batch.__new__(Batch)
        s.q, s.k, s.v, s.table, s.lens = b.q[:m], b.k, b.v, b.table[:m], b.lens[:m]
        s.check((out, lse))


def test_padded_and_empty_batches():
    import torch
    for lens in ([0, 0, 0], [0] * 300, [0] * 299 + [200]):
        b = Batch([(150, lens)], 16, 8, 2, 128, seed=14)
        for longest in (200, 16 * (b.table.shape[1])):
            b.check(b.run(True, longest=min(longest, 16 * b.table.shape[1])))
    q = torch.zeros(0, 8, 64, device="cuda", dtype=torch.bfloat16)
    pool, table = torch.zeros(2, 16, 2, 64, device="cuda", dtype=torch.bfloat16), torch.zeros(0, 2, device="cuda", dtype=torch.int32)
    out = D().decode_attention_shared(q, pool, pool, table, cu([]), cu([0]), cu([]), max_ctx_len=20)
    assert out.shape == (0, 8, 64)


def test_enough_rows_to_share_unasked():
    import torch
    b = Batch([(2100, [2110 + i for i in range(12)]), (1500, [1600, 1700])], 16, 8, 2, 64, seed=17)
    wide = torch.full((14, 200000 // 16), -1, dtype=torch.int32, device="cuda")
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    got = b.run(longest=100000, flags=0)
    b.check(got)
    assert all(torch.equal(x, y) for x, y in zip(got, b.run(longest=100000)))


def test_many_groups():
    rng = np.random.default_rng(3)
    groups = [(int(p), [int(p) + int(x) for x in rng.integers(0, 30, int(n))]) for p, n in zip(rng.integers(0, 400, 700), rng.integers(0, 4, 700))]
    b = Batch(groups, 16, 4, 2, 64, seed=15)
    b.check(b.run(True))
    assert b.status == 0


def test_refusals():
    import torch
    lib = D()
    b = Batch([(100, [130, 140])], 16, 8, 2, 64, seed=16)
    q, k, v, t, ln, st, px = b.args()
    call = lib.decode_attention_shared
    for args in ((q, k, v, t, ln, st[:0], px), (q, k, v, t, ln, st, px[:0]), (q, k, v, t, ln, st.long(), px), (q, k, v, t, ln, None, px),
                 (q, k, v, t, ln, st, None), (q, k, v, t, ln, st.cpu(), px), (q.float(), k, v, t, ln, st, px), (q, k, v[:1], t, ln, st, px),
                 (q, k, v, t, ln, st.view(1, 2), px)):
        with pytest.raises((TypeError, ValueError)):
            call(*args, max_ctx_len=140)
    for kw in (dict(max_ctx_len=100000), dict(scale=float("inf")), dict(window=-1), dict(workspace=lib.alloc_workspace(4096))):
        with pytest.raises(lib.DFlashError):
            call(*b.args(), **{**dict(max_ctx_len=140), **kw})
    with pytest.raises(lib.DFlashError):
        lib.shared_workspace_size(4, -1, 8, 2, 64, 100)
    with pytest.raises(lib.DFlashError):
        lib.shared_workspace_size(4, 1, 8, 3, 64, 100)
