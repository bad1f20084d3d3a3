"""The decode-step operators together, as a beam search uses them, against histories kept as plain lists.

Every step: room for one row per beam, rotary positions with k and v to their slots, attention over the
store, logits, selection, fork. Beside it every beam's keys and values are kept as lists; they are what
the store has to hold, bit for bit, after every fork and copy. The attention is compared with the
definition over those lists (tolerance as in test_gpu_decode_attention) and the selection with a sort.
"""
import numpy as np
import pytest

from tests import decode_ref as R
from tests.test_gpu_beam_select import check as check_beams
from tests.test_gpu_decode_attention import check as check_attention

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_beam_search_over_the_paged_store(captured):
    import torch

    import speculative_decoding_draft_rmsnorm_gb300 as D
    torch.manual_seed(0)
    reqs, w, hq, hkv, dh, ps, vocab, steps, eos = 3, 4, 8, 2, 64, 4, 500, 14, 7
    rows, pages, width = reqs * w, 200, 16
    bf16, i32 = torch.bfloat16, torch.int32
    emb = torch.randn(vocab, (hq + 2 * hkv) * dh, device="cuda").to(bf16)
    head = (0.3 * torch.randn(hq * dh, vocab, device="cuda")).to(bf16)
    freq, _ = D.rotary_frequencies(dh, 1e4)
    kp = torch.full((pages, ps, hkv, dh), float("nan"), device="cuda", dtype=bf16)
    vp = kp.clone()
    table = torch.full((rows, width), -1, device="cuda", dtype=i32)
    refs = torch.zeros(pages, device="cuda", dtype=i32)
    lens = torch.zeros(rows, device="cuda", dtype=i32)
    starts = torch.arange(rows + 1, device="cuda", dtype=i32)
    status = torch.zeros(1, device="cuda", dtype=i32)
    tokens = torch.randint(8, vocab, (reqs, 1), device="cuda").repeat(1, w).view(-1).contiguous()
    scores = torch.full((reqs, w), -float("inf"), device="cuda")
    scores[:, 0] = 0.0  # one live beam at first
    finished = torch.zeros(reqs, w, device="cuda", dtype=torch.bool)
    dec_ws = D.alloc_workspace(D.decode_workspace_size(rows, hq, hkv, dh, width * ps))
    beam_ws = D.alloc_workspace(D.beam_workspace_size(reqs, w, w, vocab, D.OUT_F32))
    page_ws = D.alloc_workspace(D.pages_workspace_size(rows, pages))
    slots, pos = torch.empty(rows, device="cuda", dtype=i32), torch.empty(rows, device="cuda", dtype=i32)
    seen, new = {}, {n: torch.empty(reqs, w, device="cuda", dtype=d) for n, d in
                     zip(("scores", "tokens", "parents", "finished"), (torch.float32, i32, i32, torch.bool))}

    def step():
        D.reserve_pages(starts, lens, table, refs, [kp, vp], num_new=rows, advance=True, slots=slots, positions=pos,
                        workspace=page_ws, status=status)
        x = emb[tokens].view(rows, hq + 2 * hkv, dh)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
        seen["q"], _ = D.rotary(q, pos, freq, k=k, v=v, k_out=kp, v_out=vp, slot=slots, status=status)
        seen["out"], seen["lse"] = D.decode_attention_paged(seen["q"], kp, vp, table, lens, max_ctx_len=width * ps,
                                                            return_lse=True, workspace=dec_ws, status=status)
        seen["logits"] = (seen["out"].view(rows, -1) @ head).float().view(reqs, w, vocab)
        D.beam_select(seen["logits"], scores, finished=finished, eos=eos, out=new, workspace=beam_ws)

    def move():
        D.fork_pages(new["parents"], lens, table, refs, status=status)
        scores.copy_(new["scores"])
        finished.copy_(new["finished"])
        tokens.copy_(new["tokens"].view(-1).clamp(min=0))

    graphs = []
    hist = [([], []) for _ in range(rows)]
    for i in range(steps):
        before = (tokens.clone(), scores.clone(), finished.clone())
        if captured and i >= 1:
            if not graphs:
                s = torch.cuda.Stream()
                for fn in (step, move):
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g, stream=s):
                        fn()
                    graphs.append(g)
            graphs[0].replay()
        else:
            step()
        torch.cuda.synchronize()
        assert status.item() == 0
        # every row's history: its own token's k (rotated alone) and v
        x = emb[before[0]].view(rows, hq + 2 * hkv, dh)
        _, k = D.rotary(None, pos, freq, k=x[:, hq:hq + hkv])
        hist = [(a + [k[r]], b + [x[r, hq + hkv:]]) for r, (a, b) in enumerate(hist)]
        ln = lens.cpu().numpy()
        assert ln.tolist() == [len(a) for a, _ in hist]
        tb = table.cpu().numpy()
        for r in range(rows):
            j = np.arange(ln[r])
            at = (torch.from_numpy(tb[r, j // ps]).cuda().long(), torch.from_numpy(j % ps).cuda())
            assert torch.equal(kp[at], torch.stack(hist[r][0])) and torch.equal(vp[at], torch.stack(hist[r][1]))
        check_attention(seen["out"], seen["lse"], seen["q"], kp, vp, table, lens)
        check_beams(new, seen["logits"], before[1], w, before[2], eos)
        held = np.bincount(tb[tb >= 0], minlength=pages)
        assert np.array_equal(refs.cpu().numpy(), held)
        par = new["parents"].view(-1).tolist()
        hist = [(list(hist[p][0]), list(hist[p][1])) if p >= 0 else ([], []) for p in par]
        if captured and i >= 1:
            graphs[1].replay()
        else:
            move()
    used = D.compact_pages(table, refs, [kp, vp])
    assert int(table.max()) < used.item() == int((refs > 0).sum())
    tb, ln = table.cpu().numpy(), lens.cpu().numpy()
    for r in range(rows):
        j = np.arange(ln[r])
        at = (torch.from_numpy(tb[r, j // ps]).cuda().long(), torch.from_numpy(j % ps).cuda())
        assert torch.equal(kp[at], torch.stack(hist[r][0]))


def test_paged_append_fills_reserved_pages():
    # the framework's own append (norm and rotary fused) into pages that reserve_pages handed out, then
    # forked rows that both append: the second one writes a copy
    import torch

    import speculative_decoding_draft_rmsnorm_gb300 as D
    torch.manual_seed(1)
    hkv, dh, ps, pages = 2, 64, 16, 12
    kp = torch.zeros(pages, ps, hkv, dh, device="cuda", dtype=torch.bfloat16)
    vp = torch.zeros_like(kp)
    table = torch.full((2, 5), -1, device="cuda", dtype=torch.int32)
    refs = torch.zeros(pages, device="cuda", dtype=torch.int32)
    lens = torch.zeros(2, device="cuda", dtype=torch.int32)
    w = torch.ones(dh, device="cuda", dtype=torch.bfloat16)
    want = [[], []]
    for counts, parent in (([20, 0], [0, 0]), ([5, 9], [0, 1]), ([16, 30], [1, 1]), ([3, 1], None)):
        starts = torch.tensor([0, counts[0], sum(counts)], device="cuda", dtype=torch.int32)
        n = sum(counts)
        k = torch.randn(n, hkv, dh, device="cuda").to(torch.bfloat16)
        v = torch.randn(n, hkv, dh, device="cuda").to(torch.bfloat16)
        status = torch.zeros(1, device="cuda", dtype=torch.int32)
        D.reserve_pages(starts, lens, table, refs, [kp, vp], num_new=n, status=status)
        D.paged_append(k, starts, lens, table, w, kp, v=v, v_pool=vp, status=status)
        assert status.item() == 0
        want[0] = want[0] + list(v[:counts[0]])
        want[1] = want[1] + list(v[counts[0]:])
        tb = table.cpu().numpy()
        for r in range(2):
            j = np.arange(len(want[r]))
            assert lens[r].item() == len(j)
            if len(j):
                at = (torch.from_numpy(tb[r, j // ps]).cuda().long(), torch.from_numpy(j % ps).cuda())
                assert torch.equal(vp[at], torch.stack(want[r]))
        if parent:
            D.fork_pages(torch.tensor(parent, device="cuda", dtype=torch.int32), lens, table, refs)
            want = [list(want[p]) for p in parent]
