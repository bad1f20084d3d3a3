"""A workspace made for the largest call does for every smaller one."""
import pytest

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("beams,out,vocab", [(8, 8, 151936), (4, 4, 20003), (1, 32, 128000), (16, 1, 300), (32, 32, 50000)])
def test_beam_workspaces_grow_with_the_call(beams, out, vocab, dtype):
    sizes = [D().beam_workspace_size(n, beams, out, vocab, dtype) for n in range(1, 257)]
    assert sizes == sorted(sizes)
    sizes = [D().beam_workspace_size(63, beams, out, v, dtype) for v in range(100, vocab, vocab // 50)]
    assert sizes == sorted(sizes)
    assert D().beam_workspace_size(63, beams, out, vocab, 0) <= D().beam_workspace_size(63, beams, out, vocab, 1)


def test_beams_of_a_smaller_batch_in_the_largest_ones_workspace():
    import torch
    n, w, vocab = 64, 8, 151936
    ws = D().alloc_workspace(D().beam_workspace_size(n, w, w, vocab))
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, w, vocab, device="cuda", generator=g).to(torch.bfloat16)
    s = -torch.rand(n, w, device="cuda", generator=g)
    for m in (64, 63, 37, 11, 10, 1):
        want, got = D().beam_select(x[:m], s[:m]), D().beam_select(x[:m], s[:m], workspace=ws)
        for k in want:
            assert torch.equal(want[k], got[k]), (m, k)


@pytest.mark.parametrize("hq,hkv", [(16, 8), (32, 8), (40, 1), (272, 2)])
@pytest.mark.parametrize("window", [0, 100])
def test_decode_workspaces_grow_with_the_call(hq, hkv, window):
    for longest in (0, 1, 16, 500, 40000):
        sizes = [D().decode_workspace_size(n, hq, hkv, 128, longest, window) for n in range(1, 400)]
        assert sizes == sorted(sizes), longest
    for n in (1, 7, 150, 1000):
        sizes = [D().decode_workspace_size(n, hq, hkv, 128, c, window) for c in range(0, 3000, 7)]
        assert sizes == sorted(sizes), n


def test_decode_of_empty_batches_in_the_largest_ones_workspace():
    import torch
    n, pools = 1000, torch.zeros(4, 16, 2, 64, device="cuda", dtype=torch.bfloat16)
    ws = D().alloc_workspace(D().decode_workspace_size(n, 8, 2, 64, 0))
    q = torch.randn(n, 8, 64, device="cuda").to(torch.bfloat16)
    table, lens = torch.full((n, 4), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    for m in (1000, 70, 1):
        out, lse = D().decode_attention_paged(q[:m], pools, pools, table[:m], lens[:m], max_ctx_len=0, workspace=ws, return_lse=True)
        assert not out.any() and bool((lse == -float("inf")).all())


def test_page_workspaces_grow_with_the_store():
    sizes = [D().pages_workspace_size(n, 5000) for n in range(1, 14000, 97)]
    assert sizes == sorted(sizes)
    sizes = [D().pages_workspace_size(300, p) for p in range(0, 100000, 997)]
    assert sizes == sorted(sizes)
