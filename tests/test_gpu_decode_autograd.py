"""The decode-step calls and autograd: nothing is recorded, so nothing is lost in silence."""
import pytest

pytestmark = pytest.mark.gpu


def D():
    import speculative_decoding_draft_rmsnorm_gb300 as lib
    return lib


def test_rotary_refuses_what_requires_a_gradient():
    import torch
    n, dh = 5, 64
    freq, _ = D().rotary_frequencies(dh)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    q, k, v = (torch.randn(n, 2, dh, device="cuda") for _ in range(3))
    store = [torch.zeros(n, 2, dh, device="cuda") for _ in range(2)]
    slot = torch.arange(n, dtype=torch.int32, device="cuda")

    def call(q=q, k=k, v=v, q_out=None, k_out=store[0], v_out=store[1]):
        return D().rotary(q, pos, freq, k=k, v=v, q_out=q_out, k_out=k_out, v_out=v_out, slot=slot)

    want = call()[0]
    for name in ("q", "k", "v", "q_out", "k_out", "v_out"):  # outputs too
        leaf = torch.randn(n, 2, dh, device="cuda", requires_grad=True)
        with pytest.raises(ValueError, match="gradient"):
            call(**{name: leaf})
        with torch.no_grad():
            call(**{name: leaf})
    leaf = q.clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        call(q=leaf * 1.0)
    assert torch.equal(call(q=leaf.detach())[0], want)
    with torch.inference_mode():
        assert torch.equal(call(q=leaf * 1.0)[0], want)


def test_the_inverse_is_the_gradient():
    import torch
    n, dh = 7, 96
    freq, amp = D().rotary_frequencies(64, scaling="parts", factor=4.0, original_len=4096)
    pos = torch.randint(0, 30000, (n,), dtype=torch.int32, device="cuda")
    x, g = torch.randn(n, 3, dh, device="cuda"), torch.randn(n, 3, dh, device="cuda")
    for inter in (False, True):
        y, _ = D().rotary(x, pos, freq, amplitude=amp, interleaved=inter)
        gx, _ = D().rotary(g, pos, freq, amplitude=amp, interleaved=inter, inverse=True)
        # <g, R x> = <R^T g, x>: each side a sum of n 3 dh products, off by 2^-22 of its terms
        left, right = (g.double() * y.double()).sum(), (gx.double() * x.double()).sum()
        size = (g.double() * y.double()).abs().sum() + (gx.double() * x.double()).abs().sum()
        assert abs(left - right) <= 2.0 ** -22 * amp * 2 * size


def test_what_a_call_writes_counts_as_changed():
    import torch
    f = dict(device="cuda")
    i = dict(device="cuda", dtype=torch.int32)
    status, freq = torch.zeros(1, **i), D().rotary_frequencies(64)[0]
    read, wrote = [], []

    def tensor(where, t):
        where.append(t)
        return t

    def check(call):
        before = [t._version for t in read], [t._version for t in wrote]
        call()
        assert [t._version for t in read] == before[0]
        assert all(t._version > v for t, v in zip(wrote, before[1]))
        read.clear(), wrote.clear()

    q, k, v = (tensor(read, torch.randn(4, 2, 64, **f)) for _ in range(3))
    ko, vo, st = tensor(wrote, torch.zeros(2, 16, 2, 64, **f)), tensor(wrote, torch.zeros(2, 16, 2, 64, **f)), tensor(wrote, status)
    qo, pos = tensor(wrote, torch.empty(4, 2, 64, **f)), tensor(read, torch.arange(4, **i))
    check(lambda: D().rotary(q, pos, freq, k=k, v=v, q_out=qo, k_out=ko, v_out=vo, slot=pos, status=st))
    x = tensor(wrote, torch.randn(4, 2, 64, **f))
    check(lambda: D().rotary(x, pos, freq, q_out=x))  # in place

    pool = tensor(read, torch.randn(2, 16, 2, 64, **f).to(torch.bfloat16))
    q = tensor(read, torch.randn(1, 4, 64, **f).to(torch.bfloat16))
    table, lens = tensor(read, torch.zeros(1, 1, **i)), tensor(read, torch.full((1,), 9, **i))
    out, lse = tensor(wrote, torch.empty(1, 4, 64, **f).to(torch.bfloat16)), tensor(wrote, torch.empty(1, 4, **f))
    ws = tensor(wrote, D().alloc_workspace(D().decode_workspace_size(1, 4, 2, 64, 16)))
    check(lambda: D().decode_attention_paged(q, pool, pool, table, lens, max_ctx_len=16, out=out, lse=lse, workspace=ws, status=st))

    x, s = tensor(read, torch.randn(2, 3, 100, **f)), tensor(read, torch.zeros(2, 3, **f))
    outs = {n: tensor(wrote, t) for n, t in D().beam_select(x, s).items()}
    check(lambda: D().beam_select(x, s, out=outs))

    pool = tensor(wrote, torch.zeros(8, 16, 64, **f))
    parent, starts = tensor(read, torch.tensor([0, 0], **i)), tensor(read, torch.tensor([0, 1, 2], **i))
    table, lens = tensor(wrote, torch.tensor([[6, -1], [-1, -1]], **i)), tensor(wrote, torch.tensor([3, 0], **i))
    refs = tensor(wrote, torch.tensor([0, 0, 0, 0, 0, 0, 1, 0], **i))
    wrote.pop(0)
    check(lambda: D().fork_pages(parent, lens, table, refs))
    wrote += [table, refs, pool]
    read += [parent, starts]
    check(lambda: D().reserve_pages(starts, lens, table, refs, [pool], num_new=2))
    wrote += [table, refs, pool]
    check(lambda: D().compact_pages(table, refs, [pool]))


def test_a_backward_pass_over_what_was_rotated_in_place_is_refused():
    import torch
    w = torch.randn(4, 2, 64, device="cuda", requires_grad=True)
    x = torch.randn(4, 2, 64, device="cuda")
    y = (w * x).sum()  # keeps x
    D().rotary(x, torch.arange(4, dtype=torch.int32, device="cuda"), D().rotary_frequencies(64)[0], q_out=x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_pools_made_in_inference_mode_may_be_written():
    import torch
    with torch.inference_mode():
        pool = torch.zeros(4, 16, 64, device="cuda")
        refs = torch.tensor([0, 0, 1, 0], dtype=torch.int32, device="cuda")
        table = torch.tensor([[2]], dtype=torch.int32, device="cuda")
    assert D().compact_pages(table, refs, [pool]).item() == 1 and table.item() == 0
