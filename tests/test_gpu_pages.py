"""dflash_fork_pages, dflash_reserve_pages and dflash_compact_pages on the GPU against the definitions
executed one sequence after the other: every integer and every copied byte is equal."""
import numpy as np
import pytest

from tests import decode_ref as R

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def cu(a):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Store:
    """A random consistent store: rows of random lengths, some sharing their first pages."""

    def __init__(self, rows, width, page, pages, seed, share=0.5, row_shape=(2, 16), pools=2, ahead=0):
        rng = np.random.default_rng(seed)
        self.page, self.rows, self.pages = page, rows, pages
        free = list(rng.permutation(pages))
        self.table = np.full((rows, width), -1, np.int32)
        self.lens = np.zeros(rows, np.int32)
        for r in range(rows):
            n = int(rng.integers(0, max(1, (width - ahead - 1) * page)))
            need = -(-n // page) + (int(rng.integers(0, ahead + 1)) if ahead else 0)
            src = int(rng.integers(0, r)) if r and rng.random() < share else -1
            held = 0
            if src >= 0:  # continues a prefix of an earlier row, its partial page perhaps included
                n = int(rng.integers(0, self.lens[src] + 1))
                need = held = -(-n // page)
                self.table[r, :held] = self.table[src, :held]
            take = min(need - held, len(free))
            if take < need - held:
                n, need = 0, 0
                self.table[r] = -1
                take, held = 0, 0
            for p in range(held, held + take):
                self.table[r, p] = free.pop()
            self.lens[r] = n
        self.refs = np.bincount(self.table[self.table >= 0], minlength=pages).astype(np.int32)
        self.pools = [rng.integers(-30000, 30000, (pages, page) + row_shape).astype(np.int16) for _ in range(pools)]

    def device(self):
        return cu(self.lens), cu(self.table), cu(self.refs), [cu(p) for p in self.pools]


def equal(t, a):
    assert np.array_equal(t.cpu().numpy(), a)


@pytest.mark.parametrize("rows,width,page,pages", [(1, 1, 16, 4), (8, 5, 16, 60), (5, 300, 1, 2000), (700, 9, 7, 5000), (3000, 3, 16, 9000)])
def test_fork_matches_definition(rows, width, page, pages):
    import torch
    rng = np.random.default_rng(rows)
    s = Store(rows, width, page, pages, seed=rows)
    lens, table, refs, _ = s.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kind in range(5):
        parent = [np.arange(rows), rng.permutation(rows), rng.integers(-1, rows, rows), np.zeros(rows), np.full(rows, -1)][kind]
        parent = parent.astype(np.int32)
        s.lens, s.table, s.refs = R.fork(parent, s.lens, s.table, s.refs)
        D().fork_pages(cu(parent), lens, table, refs, status=status)
        equal(lens, s.lens), equal(table, s.table), equal(refs, s.refs)
    assert status.item() == 0 and not s.refs.any()  # all rows freed at the end


def test_fork_reports_and_keeps_bad_parents():
    import torch
    s = Store(6, 4, 16, 60, seed=1)
    lens, table, refs, _ = s.device()
    parent = np.array([1, 6, -2, 3, -1, 0], np.int32)
    want = R.fork(parent, s.lens, s.table, s.refs)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    D().fork_pages(cu(parent), lens, table, refs, status=status)
    equal(lens, want[0]), equal(table, want[1]), equal(refs, want[2])
    assert status.item() == D().STATUS_METADATA


def reserve(s, counts, advance, n=None, pools=True, status=None):
    starts = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    n = int(starts[-1]) if n is None else n
    want = R.reserve(starts, s.lens, s.table, s.refs, s.pools if pools else [], s.page, n, advance)
    lens, table, refs, dev = s.device()
    slots, pos = D().reserve_pages(cu(starts), lens, table, refs, dev if pools else [], num_new=n, advance=advance,
                                   page_size=s.page, status=status)
    equal(lens, want[0]), equal(table, want[1]), equal(refs, want[2]), equal(slots, want[4]), equal(pos, want[5])
    for a, b in zip(dev, want[3]):
        equal(a, b)
    s.lens, s.table, s.refs, s.pools = want[0], want[1], want[2], want[3] if pools else s.pools
    return want[6], want[4]


@pytest.mark.parametrize("rows,width,page,pages,most", [(1, 4, 16, 6, 9), (8, 12, 16, 200, 3), (40, 6, 5, 400, 12), (300, 40, 16, 9000, 70),
                                                        (1000, 5, 16, 9000, 1), (20, 100, 1, 3000, 30), (6, 9, 24, 40000, 24)])
def test_reserve_matches_definition(rows, width, page, pages, most):
    import torch
    rng = np.random.default_rng(rows)
    s = Store(rows, width, page, pages, seed=rows + 1, ahead=1)
    for step in range(3):
        counts = rng.integers(0, most + 1, rows)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        bad, _ = reserve(s, counts, advance=step != 1, status=status)
        assert status.item() == (D().STATUS_METADATA if bad else 0)


def test_reserve_when_pages_run_out_and_tables_fill():
    import torch
    s = Store(10, 6, 4, 24, seed=5, share=0.6)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    seen = []
    for _ in range(6):
        bad, slots = reserve(s, np.full(10, 3), advance=True, status=status)
        seen.append(bad)
    assert any(seen) and status.item() == D().STATUS_METADATA
    full = Store(2, 3, 4, 24, seed=6, share=0.0)
    full.lens[:] = 0
    full.table[:] = -1
    full.refs[:] = 0
    bad, slots = reserve(full, [13, 12], advance=True)  # 13 rows do not fit 3 pages of 4
    assert bad and (slots[:13] == -1).all() and (slots[13:] >= 0).all()


def test_reserve_bad_metadata_changes_nothing():
    import torch
    for starts in ([1, 0, 2], [-1, 1, 2], [0, 1, 9]):
        s = Store(2, 4, 4, 24, seed=7)
        lens, table, refs, dev = s.device()
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        slots, pos = D().reserve_pages(cu(np.array(starts, np.int32)), lens, table, refs, dev, num_new=4, advance=True, status=status)
        equal(lens, s.lens), equal(table, s.table), equal(refs, s.refs)
        assert bool((slots == -1).all()) and not bool(pos.any()) and status.item() == D().STATUS_METADATA
    s = Store(5, 4, 4, 40, seed=8, share=0.0)
    s.lens[:] = [5, 5, -3, 5, 6]
    s.table[:, :2] = [[0, 1], [2, 99], [4, 5], [6, -1], [7, 8]]
    s.table[:, 2:] = -1
    s.refs[:] = 0
    s.refs[[0, 1, 2, 4, 5, 6, 7, 8]] = 1
    s.refs[8] = 0  # row 4 names a page that counts as free
    bad, slots = reserve(s, [4, 4, 4, 4, 4], advance=True)
    assert bad and (slots[:4] >= 0).all() and (slots[4:] == -1).all()


def test_reserve_rows_outside_the_starts_and_without_pools():
    s = Store(3, 6, 8, 40, seed=9)
    starts = np.array([2, 3, 3, 7], np.int32)
    want = R.reserve(starts, s.lens, s.table, s.refs, [], 8, 10, False)
    lens, table, refs, _ = s.device()
    slots, pos = D().reserve_pages(cu(starts), lens, table, refs, [], num_new=10, page_size=8)
    equal(lens, want[0]), equal(table, want[1]), equal(refs, want[2]), equal(slots, want[4]), equal(pos, want[5])


@pytest.mark.parametrize("rows,width,page,pages,keep", [(1, 1, 16, 4, 1.0), (8, 12, 16, 200, 0.6), (50, 40, 4, 3000, 0.4), (4, 9, 24, 40000, 1.0),
                                                        (20, 6, 2, 1024, 0.0), (100, 30, 16, 1025, 0.7)])
def test_compact_matches_definition(rows, width, page, pages, keep):
    import torch
    rng = np.random.default_rng(pages)
    s = Store(rows, width, page, pages, seed=pages)
    parent = np.where(rng.random(rows) < keep, np.arange(rows), -1)
    s.lens, s.table, s.refs = R.fork(parent, s.lens, s.table, s.refs)
    lens, table, refs, dev = s.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = R.compact(s.table, s.refs, s.pools)
    used = D().compact_pages(table, refs, dev, status=status)
    assert used.item() == want[3] and status.item() == 0
    equal(table, want[0]), equal(refs, want[1])
    for a, b in zip(dev, want[2]):
        equal(a, b)
    assert (want[1][:want[3]] > 0).all() and not want[1][want[3]:].any()
    used = D().compact_pages(table, refs, dev)  # again: nothing moves
    equal(table, want[0]), equal(refs, want[1])
    for a, b in zip(dev, want[2]):
        equal(a, b)


def test_compact_reports_entries_that_are_no_pages():
    import torch
    s = Store(3, 4, 4, 40, seed=11)
    lens, table, refs, dev = s.device()
    table[2, 3] = 1000
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    D().compact_pages(table, refs, dev, status=status)
    assert status.item() == D().STATUS_METADATA and table[2, 3].item() == 1000


def test_strided_tables_and_a_captured_step():
    # a table inside a wider one; fork and reserve captured once and replayed as the state moves on
    import torch
    s = Store(12, 20, 4, 300, seed=12, share=0.3)
    wide = torch.full((12, 33), 555, dtype=torch.int32, device="cuda")
    table = wide[:, 5:25]
    table.copy_(cu(s.table))
    lens, _, refs, dev = s.device()
    parent = cu(np.arange(12, dtype=np.int32))
    starts = cu(np.arange(13, dtype=np.int32))
    slots = torch.empty(12, dtype=torch.int32, device="cuda")
    pos = torch.empty(12, dtype=torch.int32, device="cuda")
    ws = D().alloc_workspace(D().pages_workspace_size(12, 300))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        D().fork_pages(parent, lens, table, refs)
        D().reserve_pages(starts, lens, table, refs, dev, num_new=12, advance=True, slots=slots, positions=pos, workspace=ws)
    rng = np.random.default_rng(13)
    for _ in range(9):
        par = rng.integers(0, 12, 12).astype(np.int32)
        parent.copy_(torch.from_numpy(par))
        g.replay()
        s.lens, s.table, s.refs = R.fork(par, s.lens, s.table, s.refs)
        s.lens, s.table, s.refs, s.pools, ws_, wp, _ = R.reserve(np.arange(13), s.lens, s.table, s.refs, s.pools, 4, 12, True)
        equal(lens, s.lens), equal(table, s.table), equal(refs, s.refs), equal(slots, ws_), equal(pos, wp)
        for a, b in zip(dev, s.pools):
            equal(a, b)
    assert bool((wide[:, :5] == 555).all()) and bool((wide[:, 25:] == 555).all())


def test_refusals():
    import torch
    d = D()
    s = Store(3, 4, 4, 40, seed=14)
    lens, table, refs, dev = s.device()
    par, starts = cu(np.arange(3, dtype=np.int32)), cu(np.arange(4, dtype=np.int32))
    small = torch.empty(256, dtype=torch.uint8, device="cuda")
    for exc, fn in [
        (TypeError, lambda: d.fork_pages(par.long(), lens, table, refs)),
        (ValueError, lambda: d.fork_pages(par[:2], lens, table, refs)),
        (ValueError, lambda: d.fork_pages(par, lens, table.t(), refs)),
        (d.DFlashError, lambda: d.fork_pages(lens, lens, table, refs)),
        (ValueError, lambda: d.fork_pages(par, lens.cpu(), table, refs)),
        (ValueError, lambda: d.reserve_pages(starts, lens, table, refs, [dev[0][:-1]], num_new=3)),
        (ValueError, lambda: d.reserve_pages(starts, lens, table, refs, [], num_new=3)),
        (ValueError, lambda: d.reserve_pages(starts, lens, table, refs, [dev[0], dev[1][..., :8].contiguous()], num_new=3)),
        (ValueError, lambda: d.reserve_pages(starts[:3], lens, table, refs, dev, num_new=3)),
        (ValueError, lambda: d.reserve_pages(starts, lens, table, refs, dev, num_new=-1)),
        (d.DFlashError, lambda: d.reserve_pages(starts, lens, table, refs, dev, num_new=3, workspace=small)),
        (d.DFlashError, lambda: d.reserve_pages(starts, lens, table, refs, [dev[0][..., :3].contiguous()], num_new=3)),
        (TypeError, lambda: d.compact_pages(table, refs.long(), dev)),
        (d.DFlashError, lambda: d.compact_pages(table, refs, dev, workspace=small)),
    ]:
        with pytest.raises(exc):
            fn()
    with pytest.raises(d.DFlashError):
        d.fork_pages(torch.zeros(16385, dtype=torch.int32, device="cuda"), torch.zeros(16385, dtype=torch.int32, device="cuda"),
                     torch.zeros(16385, 1, dtype=torch.int32, device="cuda"), refs)
