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
