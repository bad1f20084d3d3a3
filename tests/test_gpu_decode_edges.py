"""Decode-step calls at the ends of what they take: the largest and oddest shapes, two calls at once, the same
thing named twice. Tolerances are those of the operators' own tests."""
import numpy as np
import pytest

from tests import decode_ref as R
from tests import test_gpu_beam_select as B
from tests import test_gpu_decode_attention as A
from tests import test_gpu_pages as P
from tests import test_gpu_rotary as T

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


@pytest.mark.parametrize("f32", [False, True])
def test_rotary_of_head_major_and_broadcast_rows(f32):
    import torch
    dtype = torch.float32 if f32 else torch.bfloat16
    n, h, dh = 37, 6, 96
    freq, _ = D().rotary_frequencies(64)
    x = torch.randn(h, n, dh, device="cuda").to(dtype).transpose(0, 1)
    pos = torch.randint(-1000, 1000, (n,), device="cuda", dtype=torch.int32)
    out = torch.zeros(h, n, dh, device="cuda", dtype=dtype).transpose(0, 1)
    D().rotary(x, pos, freq, q_out=out)
    T.check(out, x, pos, freq)
    got, _ = D().rotary(x[:1].expand(n, h, dh), pos, freq)  # one row at every position
    T.check(got, x[:1].expand(n, h, dh), pos, freq)
    inner = torch.zeros(n, h, dh + 8, device="cuda", dtype=dtype)
    D().rotary(x, pos, freq, q_out=inner[:, :, :dh])
    T.check(inner[:, :, :dh], x, pos, freq)
    assert not inner[:, :, dh:].any()
    for bad in (out[:1].expand(n, h, dh), out[:, :1].expand(n, h, dh)):  # rows or heads on top of one another
        with pytest.raises(D().DFlashError):
            D().rotary(x, pos, freq, q_out=bad)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("hq,hkv,dh", [(272, 2, 64), (129, 1, 128), (48, 2, 128)])
def test_decode_with_groups_of_many_heads(hq, hkv, dh, f32):
    lens = [3000, 1, 0, 777, 16]
    q = A.queries(len(lens), hq, dh)
    k, v, table, ln = A.store(lens, 16, hkv, dh, seed=20)
    out, lse = A.attend(q, k, v, table, ln, f32=f32)
    A.check(out, lse, q, k, v, table, ln)


def test_decode_with_a_page_named_twice_and_a_broadcast_query():
    import torch
    k, v, table, ln = A.store([64, 640], 16, 2, 64, seed=21)
    table[1, 5:20] = table[1, 4]
    q = A.queries(1, 8, 64).expand(2, 8, 64)
    out, lse = A.attend(q, k, v, table, ln, f32=True)
    A.check(out, lse, q, k, v, table, ln)
    torch.cuda.synchronize()


@pytest.mark.parametrize("lens", [[0, 0, 0], [0] * 200, [0] * 199 + [5]])
def test_decode_of_a_padded_batch(lens):
    q = A.queries(len(lens), 8, 128)
    k, v, table, ln = A.store(lens, 16, 2, 128, seed=22)
    for longest in (32, 30000):
        import torch
        wide = torch.full((len(lens), 2000), -1, dtype=torch.int32, device="cuda")
        wide[:, :table.shape[1]] = table
        out, lse = A.attend(q, k, v, wide, ln, longest=longest)
        A.check(out, lse, q, k, v, table, ln)


def test_two_calls_at_once():
    import torch
    lens = [5000, 40, 900, 2200]
    sets = []
    for i in range(2):
        k, v, table, ln = A.store(lens, 16, 4, 128, seed=30 + i)
        x, s = B.draw(6, 4, 50000, False, seed=30 + i)
        sets.append((A.queries(4, 32, 128, seed=i), k, v, table, ln, x, s))
    want = [(A.attend(*z[:5]), D().beam_select(*z[5:])) for z in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    graphs = []
    for z, st in zip(sets, streams):
        st.wait_stream(torch.cuda.current_stream())
        out = torch.empty(4, 32, 128, device="cuda", dtype=torch.bfloat16)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            D().decode_attention_paged(*z[:5], max_ctx_len=5000, out=out)
        graphs.append((g, out))
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for z, st, (g, out) in zip(sets, streams, graphs):
            with torch.cuda.stream(st):
                g.replay()
                got.append((A.attend(*z[:5], longest=5000), D().beam_select(*z[5:])))
        torch.cuda.synchronize()
        for (a, b), (wa, wb), (_, out) in zip(got, want, graphs):
            assert torch.equal(a[0], wa[0]) and torch.equal(a[1], wa[1]) and torch.equal(out, wa[0])
            assert all(torch.equal(b[n], wb[n]) for n in wb)


@pytest.mark.parametrize("f32", [False, True])
def test_beams_of_the_largest_vocabulary(f32):
    import torch
    vocab = (1 << 26) - 1
    g = torch.Generator(device="cuda").manual_seed(40)
    x = torch.empty(1, 1, vocab, device="cuda", dtype=torch.float32 if f32 else torch.bfloat16).normal_(generator=g)
    top = torch.tensor([vocab - 1, 7, vocab // 2, 0], device="cuda")
    x[0, 0, top] = torch.tensor([9.0, 8.0, 8.0, 7.0], device="cuda").to(x.dtype)
    s = torch.full((1, 1), -2.5, device="cuda")
    got = D().beam_select(x, s, beams_out=4, eos=7)
    assert got["tokens"].tolist() == [[vocab - 1, 7, vocab // 2, 0]] and got["parents"].tolist() == [[0] * 4]
    assert got["finished"].tolist() == [[False, True, False, False]]
    lse = torch.logsumexp(x.double(), -1).item()
    want = np.array([9.0, 8.0, 8.0, 7.0]) - 2.5 - lse
    tol = 2.0 ** -24 * np.abs(want) + 2.0 ** -21 + (64 + vocab / 2048) * 2.0 ** -24
    assert np.all(np.abs(got["scores"][0].double().cpu().numpy() - want) <= tol)
    with pytest.raises(D().DFlashError):
        D().beam_select(torch.empty(1, 1, vocab + 1, device="cuda", dtype=torch.bfloat16), s)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("n,w,k,vocab", [
    (140, 16, 16, 242), (12, 2, 16, 664), (256, 5, 16, 97),        # rows read one by one
    (9, 4, 32, 1024), (9, 4, 32, 1025), (3, 8, 17, 1031),          # ... and just not; 64 groups
    (2, 16, 32, 20011), (1, 1, 32, 60000), (1, 1, 31, 128001),     # many lists of many places
    (100, 1, 1, 20000), (75, 4, 4, 20000), (200, 4, 4, 5000),      # rows cut each for itself, or laid end to end
])
def test_beams_of_every_cut(n, w, k, vocab, f32):
    import torch
    x, s = B.draw(n, w, vocab, f32, seed=vocab + k)
    B.check(D().beam_select(x, s, beams_out=k), x, s, k)
    x = x[:2].round()  # few distinct values
    x[0, 0] = 0.5
    x[-1, 0] = torch.sort(x[-1, 0]).values
    s = -torch.arange(w, device="cuda", dtype=torch.float32).repeat(x.shape[0], 1)  # no two beams of equal scores
    B.check(D().beam_select(x, s, beams_out=k), x, s, k)


def test_as_many_beams_as_there_may_be_over_a_wide_vocabulary():
    x, s = B.draw(1, 32, 300007, False, seed=41)
    B.check(D().beam_select(x, s), x, s, 32)


def test_the_most_table_rows():
    import torch
    rows = 14000
    s = P.Store(rows, 3, 16, 40000, seed=50, ahead=1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.reserve(s, np.ones(rows, int), advance=True, status=status)
    lens, table, refs, pools = s.device()
    parent = np.random.default_rng(51).integers(-1, rows, rows).astype(np.int32)
    want = R.fork(parent, s.lens, s.table, s.refs)
    D().fork_pages(P.cu(parent), lens, table, refs, status=status)
    P.equal(lens, want[0]), P.equal(table, want[1]), P.equal(refs, want[2])
    wt, wr, wp, used = R.compact(want[1], want[2], s.pools)
    assert D().compact_pages(table, refs, pools, status=status).item() == used and status.item() == 0
    P.equal(table, wt), P.equal(refs, wr), P.equal(pools[0], wp[0])
    more = torch.full((rows + 1, 3), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(D().DFlashError):
        D().fork_pages(torch.zeros(rows + 1, dtype=torch.int32, device="cuda"), torch.zeros(rows + 1, dtype=torch.int32, device="cuda"), more, refs)


def test_more_pages_than_pieces_of_the_smallest_size():
    # above 1024 x 1024 pages a piece of the counts grows
    import torch
    pages = 1500007
    s = P.Store(40, 2000, 1, pages, seed=52, row_shape=(8,), pools=1, ahead=1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    P.reserve(s, np.full(40, 60), advance=True, status=status)
    lens, table, refs, pools = s.device()
    wt, wr, wp, used = R.compact(s.table, s.refs, s.pools)
    assert D().compact_pages(table, refs, pools, status=status).item() == used and status.item() == 0
    P.equal(table, wt), P.equal(refs, wr)
    P.equal(pools[0][:used], wp[0][:used])


def test_a_pool_listed_twice_and_pools_without_pages():
    import torch
    s = P.Store(8, 12, 16, 200, seed=53)
    lens, table, refs, pools = s.device()
    wt, wr, wp, used = R.compact(s.table, s.refs, s.pools)
    assert D().compact_pages(table, refs, [pools[0], pools[1], pools[0]]).item() == used
    P.equal(table, wt), P.equal(refs, wr)
    for a, b in zip(pools, wp):
        P.equal(a[:used], b[:used])
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    empty = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots, pos = D().reserve_pages(starts, torch.zeros(1, dtype=torch.int32, device="cuda"), empty, none, [], num_new=2, page_size=16,
                                   status=status)
    assert slots.tolist() == [-1, -1] and status.item() == D().STATUS_METADATA and bool((empty == -1).all())
    assert D().compact_pages(empty, none, []).item() == 0
