"""The operators of a step over a shared prompt together, as a decoder layer uses them.

A prompt is stored once for every request; its samples fork from it, and in every step each of them makes room for a row,
normalises its state, projects it, turns q and k by positions on three axes (k and v to their slots), and attends. Each
operator is compared with its own definition on what it was given, by the checks of its own tests, and the attention also
with that of calls in which every sequence reads its own rows.
"""
import numpy as np
import pytest

from tests.test_gpu_rms_norm import check as check_norm
from tests.test_gpu_rotary_axes import check as check_axes
from tests.test_gpu_shared_attention import check as check_attention
from tests.test_gpu_shared_prefixes import define as define_prefixes

pytestmark = pytest.mark.gpu


class Step:
    """Requests of w samples each; state [rows, d] is the residual stream."""

    def __init__(self, D, prompts, w, hq, hkv, dh, ps, seed=0, window=0, stream=None):
        import torch
        self.D, self.w, self.hq, self.hkv, self.dh, self.ps, self.window, self.stream = D, w, hq, hkv, dh, ps, window, stream
        g = torch.Generator(device="cuda").manual_seed(seed)
        i32 = dict(dtype=torch.int32, device="cuda")
        rows, d = len(prompts) * w, hq * dh
        self.rows, self.width = rows, -(-(max(prompts) + 40) // ps)
        pages = sum(-(-p // ps) for p in prompts) + rows * (40 // ps + 3)
        self.kp, self.vp = (torch.full((pages, ps, hkv, dh), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
        self.table = torch.full((rows, self.width), -1, **i32)
        self.lens, self.refs = torch.zeros(rows, **i32), torch.zeros(pages, **i32)
        self.starts, self.each = torch.arange(0, rows + 1, w, **i32), torch.arange(rows + 1, **i32)
        self.status = torch.zeros(1, **i32)
        self.freq, _ = D.rotary_frequencies(dh)
        self.axes = D.rotary_sections((dh // 8, 3 * dh // 16, 3 * dh // 16), interleaved=True)
        self.three = torch.tensor([[1], [2], [0]], **i32)  # axis a's position is pos * three[a] + three[a] // 2
        self.wn = (1 + 0.1 * torch.randn(d, device="cuda", generator=g)).to(torch.bfloat16)
        self.proj = (0.05 * torch.randn(d, (hq + 2 * hkv) * dh, device="cuda", generator=g)).to(torch.bfloat16)
        self.state = torch.randn(rows, d, device="cuda", generator=g).to(torch.bfloat16)
        self.out = torch.randn(rows, d, device="cuda", generator=g).to(torch.bfloat16)
        self.slots, self.pos = torch.empty(rows, **i32), torch.empty(rows, **i32)
        self.page_ws = D.alloc_workspace(D.pages_workspace_size(rows, pages))
        self.most = self.width * ps
        self.ws = D.alloc_workspace(D.shared_workspace_size(rows, len(prompts), hq, hkv, dh, self.most, window))
        # the prompts: rows of each request's first sample, which the others fork
        count = [p if r % w == 0 else 0 for p, r in ((prompts[r // w], r) for r in range(rows))]
        loc = torch.tensor(np.concatenate(([0], np.cumsum(count))), **i32)
        slots, _ = D.reserve_pages(loc, self.lens, self.table, self.refs, [self.kp, self.vp], num_new=sum(count), advance=True)
        for pool in (self.kp, self.vp):
            pool.view(-1, hkv, dh)[slots.long()] = torch.randn(sum(count), hkv, dh, device="cuda", generator=g).to(torch.bfloat16)
        self.parents = torch.arange(rows, **i32) // w * w
        D.fork_pages(self.parents, self.lens, self.table, self.refs, status=self.status)

    def __call__(self):
        D, hq, hkv, dh, at = self.D, self.hq, self.hkv, self.dh, dict(status=self.status, stream=self.stream)
        D.reserve_pages(self.each, self.lens, self.table, self.refs, [self.kp, self.vp], num_new=self.rows, advance=True, slots=self.slots,
                        positions=self.pos, workspace=self.page_ws, **at)
        self.prefixes = D.shared_prefixes(self.table, self.lens, self.starts, page_size=self.ps, **at)
        self.given = self.out.clone(), self.state.clone()
        self.normed = D.rms_norm(self.out, self.wn, residual=self.state, residual_out=self.state, **at)
        self.x = (self.normed[0] @ self.proj).view(self.rows, hq + 2 * hkv, dh)
        self.grid = self.pos.view(1, -1) * self.three + self.three // 2
        self.q, _ = D.rotary_axes(self.x[:, :hq], self.grid, self.axes, self.freq, k=self.x[:, hq:hq + hkv], k_out=self.kp, v=self.x[:, hq + hkv:],
                                  v_out=self.vp, slot=self.slots, **at)
        out, self.lse = D.decode_attention_shared(self.q, self.kp, self.vp, self.table, self.lens, self.starts, self.prefixes, max_ctx_len=self.most,
                                                  return_lse=True, workspace=self.ws, window=self.window, flags=D.FLAG_FORCE_SHARE, **at)
        self.out.copy_(out.view(self.rows, -1))

    def check(self, expect_shared=True):
        import torch
        torch.cuda.synchronize()
        hq, hkv = self.hq, self.hkv
        assert self.status.item() == 0
        table, lens = self.table.cpu().numpy(), self.lens.cpu().numpy()
        got = self.prefixes.tolist()
        assert got == define_prefixes(table, lens, self.starts.tolist(), self.ps)
        assert not expect_shared or min(got) >= 64
        check_norm((self.normed[0], self.state, None), *self.given, self.wn)
        check_axes(self.q, self.x[:, :hq], self.grid, self.axes, self.freq)
        for pool, want in ((self.kp, None), (self.vp, self.x[:, hq + hkv:])):
            rows = pool.view(-1, hkv, self.dh)[self.slots.long()]
            if want is None:
                check_axes(rows, self.x[:, hq:hq + hkv], self.grid, self.axes, self.freq)
            else:
                assert torch.equal(rows, want)
        b = type("", (), {})()
        b.q, b.k, b.v, b.table, b.lens = self.q, self.kp, self.vp, self.table, lens
        check_attention((self.out.view_as(self.q), self.lse), b, self.window)
        own = self.D.decode_attention_paged(self.q, self.kp, self.vp, self.table, self.lens, max_ctx_len=self.most, window=self.window, return_lse=True)
        check_attention(own, b, self.window)


def make(**kw):
    import speculative_decoding_draft_rmsnorm_gb300 as D
    return Step(D, **kw)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("window", [0, 90])
def test_samples_of_shared_prompts(captured, window):
    import torch
    s = make(prompts=[200, 128, 333], w=4, hq=8, hkv=2, dh=64, ps=16, window=window)
    g = None
    for i in range(20):  # past the end of a page
        if i == 9:  # the samples of every request go on from its second one: what that wrote is shared too
            s.parents.copy_(torch.arange(s.rows, device="cuda", dtype=torch.int32) // s.w * s.w + 1)
            s.D.fork_pages(s.parents, s.lens, s.table, s.refs, status=s.status)
        if captured and i >= 1:
            if g is None:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    s()
            g.replay()
        else:
            s()
        if i in (0, 1, 8, 9, 10, 19):
            s.check()


def test_two_graphs_in_turn_over_one_workspace():
    import torch
    a, b = (make(prompts=p, w=5, hq=16, hkv=2, dh=128, ps=ps, seed=len(p)) for p, ps in (([300, 150], 16), ([700, 90], 24)))
    ws = max(a.ws, b.ws, key=lambda t: t.numel())
    a.ws = b.ws = ws
    graphs = []
    for s in (a, b):
        s()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s()
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, (a, b)):
            g.replay()
        for s in (a, b):
            s.check()


def test_on_another_stream():
    import torch
    st = torch.cuda.Stream()
    s = make(prompts=[260, 70], w=3, hq=4, hkv=4, dh=128, ps=16)
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        s.stream = st
        for _ in range(3):
            s()
    st.synchronize()
    s.check()


def test_wide_samples_of_one_prompt():
    # 70 samples, 560 rows of a product; 8-row pages, which a prefix ends in the middle of a tile with
    s = make(prompts=[500], w=70, hq=16, hkv=2, dh=64, ps=8)
    for _ in range(9):
        s()
    s.check()
