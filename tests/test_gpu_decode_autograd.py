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
