"""dflash_shared_prefixes on the GPU against its definition, exactly."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def cu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def define(table, lens, starts, page):
    out = []
    for a, b in zip(starts[:-1], starts[1:]):
        ok = 0 <= a <= b <= len(lens)
        live = [r for r in range(a, b) if 0 < lens[r] <= table.shape[1] * page] if ok else []
        c = 0
        while live and c < table.shape[1] and table[live[0], c] >= 0 and all(table[r, c] == table[live[0], c] for r in live):
            c += 1
        out.append(min([c * page] + [int(lens[r]) for r in live]) if live else 0)
    return out


def draw(starts, width, page, seed, depth):
    """Tables whose groups share about `depth` entries."""
    rng = np.random.default_rng(seed)
    n = starts[-1]
    table, lens = rng.integers(0, 1 << 30, (n, width)), rng.integers(1, width * page + 1, n)
    for a, b in zip(starts[:-1], starts[1:]):
        d = int(rng.integers(0, depth + 1))
        table[a:b, :d] = rng.integers(0, 1 << 30, d)
        lens[a:b] = np.maximum(lens[a:b], min(width * page, int(rng.integers(1, depth * page + 2))))
    return table.astype(np.int32), lens.astype(np.int32)


@pytest.mark.parametrize("starts,width,page", [([0, 1], 1, 16), ([0, 4], 50, 16), ([0, 3, 3, 10, 11], 700, 24), (list(range(0, 257, 8)), 300, 16),
                                               ([0, 256], 2100, 16), ([0, 0, 0], 4, 16), ([0, 700], 513, 1), (list(range(400)), 9, 64),
                                               ([0, 1200], 40, 5), ([0, 2, 40], 5000, 128)])
def test_matches_definition(starts, width, page):
    import torch
    for seed in range(4):
        table, lens = draw(starts, width, page, seed, [1, width // 2, width, width][seed])
        if seed >= 2:
            lens[np.random.default_rng(seed).random(len(lens)) < 0.3] = 0
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = D().shared_prefixes(cu(table), cu(lens), cu(starts), page_size=page, status=status)
        assert got.tolist() == define(table, lens, starts, page) and status.item() == 0
        wide = cu(np.full((len(lens), width + 7), -5))
        wide[:, 3:3 + width] = cu(table)
        assert torch.equal(D().shared_prefixes(wide[:, 3:3 + width], cu(lens), cu(starts), page_size=page), got)


@pytest.mark.parametrize("at", [0, 1, 31, 32, 511, 512, 513, 1999])
def test_one_difference(at):
    table = np.tile(np.arange(2000, dtype=np.int32), (37, 1))
    lens = np.full(37, 2000 * 16 - 3, np.int32)
    for row, value in ((36, 77777), (17, -1), (0, 5555)):
        t = table.copy()
        t[row, at] = value
        got = D().shared_prefixes(cu(t), cu(lens), cu([0, 37]), page_size=16)
        assert got.tolist() == [min(at * 16, 2000 * 16 - 3)]
    t = table.copy()
    t[:, at] = -1  # the same everywhere, but no page
    assert D().shared_prefixes(cu(t), cu(lens), cu([0, 37]), page_size=16).tolist() == [at * 16]
    lens[5] = 0  # a sequence that is not there does not count
    t[5] = 99
    t[:, at] = at
    t[5, at] = 99
    assert D().shared_prefixes(cu(t), cu(lens), cu([0, 37]), page_size=16).tolist() == [2000 * 16 - 3]


def test_bad_metadata_is_reported():
    import torch
    table, lens = np.tile(np.arange(10, dtype=np.int32), (6, 1)), np.array([20, -1, 161, 160, 30, 40], np.int32)
    for starts in ([0, 3, 6], [0, 7, 6], [-1, 3, 6], [4, 2, 6]):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = D().shared_prefixes(cu(table), cu(lens), cu(starts), page_size=16, status=status)
        assert got.tolist() == define(table, lens, starts, 16) and status.item() == D().STATUS_METADATA, starts


def test_refusals_streams_and_capture():
    import torch
    lib = D()
    table, lens = draw([0, 4, 9], 40, 16, 1, 40)
    t, ln, st = cu(table), cu(lens), cu([0, 4, 9])
    for args, kw in (((t, ln, st), dict(page_size="x")), ((t, ln[:8], st), {}), ((t[0], ln, st), {}), ((t, ln, st[:0]), {}), ((t.long(), ln, st), {}),
                     ((t, ln, st.cpu()), {}), ((t, None, st), {}), ((t, ln, st), dict(out=ln)), ((t.t(), ln, st), {}),
                     ((t, ln, st), dict(out=torch.zeros(2, device="cuda")))):
        with pytest.raises((TypeError, ValueError)):
            lib.shared_prefixes(*args, **{**dict(page_size=16), **kw})
    for kw in (dict(page_size=0), dict(out=ln[:2]), dict(out=st[1:]), dict(out=t[0, :2])):
        with pytest.raises(lib.DFlashError):
            lib.shared_prefixes(t, ln, st, **{**dict(page_size=16), **kw})
    out, g = torch.empty(2, dtype=torch.int32, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lib.shared_prefixes(t, ln, st, page_size=16, out=out)
    table2, lens2 = draw([0, 4, 9], 40, 16, 2, 40)
    t.copy_(cu(table2)), ln.copy_(cu(lens2))
    g.replay()
    assert out.tolist() == define(table2, lens2, [0, 4, 9], 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.shared_prefixes(t, ln, st, page_size=16, stream=side)
    side.synchronize()
    assert torch.equal(got, out) and out._version >= 1
