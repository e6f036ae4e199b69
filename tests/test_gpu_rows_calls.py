"""Calls of the row operators that their documentation allows beside the ordinary ones."""
import pytest
import torch

pytestmark = pytest.mark.gpu

q = pytest.importorskip("quantized_mixture_experts_grouped_b200")


def room_for(gb):
    if torch.cuda.mem_get_info()[0] < gb * 2**30:
        pytest.skip(f"needs {gb} GB of device memory")


# rows that take more than 65535 blocks along their columns: single values, words of one chunk per
# thread (more than four choices in 16 bits), words of two
@pytest.mark.parametrize("H,k", [(2**27 + 1, 1), (2**27 + 8, 8), (2**28 + 8, 1)])
def test_very_wide_rows(H, k):
    """Small whole numbers: every product and sum is exact."""
    room_for(16)
    g = torch.Generator(device="cuda").manual_seed(k)
    yp = torch.randint(-8, 9, (k, H), generator=g, device="cuda", dtype=torch.int8).bfloat16()
    inv = torch.arange(k, dtype=torch.int32, device="cuda").view(1, k)
    wts = torch.full((1, k), 0.5, device="cuda")
    out = torch.full((1, H), 77.0, dtype=torch.bfloat16, device="cuda")
    total = yp.sum(0, keepdim=True, dtype=torch.float32)
    q.moe_combine(yp, inv, wts, out)
    assert torch.equal(out, (total * 0.5).bfloat16())
    q.moe_dispatch_backward(yp, inv, out)
    assert torch.equal(out, total.bfloat16())
    if k == 1:
        i32 = dict(dtype=torch.int32, device="cuda")
        xp = torch.full_like(yp, 77.0)
        q.moe_dispatch(yp, inv, 1, torch.empty(1, **i32), torch.empty(2, **i32), torch.empty(1, **i32),
                       torch.empty_like(inv), xp)
        assert torch.equal(xp, yp)
        q.moe_combine_backward(yp, None, inv, wts, dyp=xp)
        assert torch.equal(xp, (yp.float() * 0.5).bfloat16())


def test_most_tokens():
    """2^31 - 1 tokens of one value each, several to a block: every one is written."""
    room_for(48)
    T = 2**31 - 1
    row = torch.full((1, 1), 3.0, dtype=torch.bfloat16, device="cuda").expand(T, 1)
    out = torch.full((T, 1), 77.0, dtype=torch.bfloat16, device="cuda")

    def all_are(value):
        return all(bool((part == value).all()) for part in out.split(2**28))
    q.moe_norm_pre(row, None, 1e-5, out)
    assert all_are(1.0)
    q.moe_norm_post(row, row, out, 1e-5, alpha=2.0)
    assert all_are(7.0)
    zeros = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    ones = torch.ones((T, 1), device="cuda")
    q.moe_combine(row, zeros, ones, out)
    assert all_are(3.0)
    q.moe_route_topk_backward(zeros, ones, ones, out)          # 1 * (1 - 1 * 1)
    assert all_are(0.0)


def test_router_gradient_with_dropped_choices():
    """Choices dropped after the router, by -1 in a copy of its ids: with the router's own ids the logits'
    gradient is autograd's, a dropped choice's logit included."""
    import rows_ref as ref
    g = torch.Generator().manual_seed(14)
    T, E, k, H = 40, 16, 4, 64
    logits = torch.randn((T, E), generator=g).bfloat16()
    idx, wts = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    q.moe_route_topk(logits.cuda(), k, idx, wts)
    kept = torch.where(torch.rand((T, k), generator=g).cuda() < 0.3, -1, idx)
    x, dout = torch.randn((T, H), generator=g).cuda(), torch.randn((T, H), generator=g).cuda()
    i32 = dict(dtype=torch.int32, device="cuda")
    inv, xp = torch.empty((T, k), **i32), torch.zeros((T * k, H), device="cuda")
    q.moe_dispatch(x, kept, E, torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32), inv, xp)
    scale = torch.randn(T * k, 1, generator=g).cuda()        # the experts: a factor of each row
    yp, dwts, dlogits = xp * scale, torch.empty_like(wts), torch.empty((T, E), device="cuda")
    q.moe_combine_backward(dout, yp, inv, wts, dwts=dwts)
    q.moe_route_topk_backward(idx, wts, dwts, dlogits)
    z = logits.double().requires_grad_()
    w = torch.softmax(z.gather(1, idx.cpu().long()), 1)
    rows = torch.where((inv >= 0)[:, :, None], yp[inv.clamp(min=0).long()], 0.0).cpu().double()
    ((w[:, :, None] * rows).sum(1) * dout.cpu().double()).sum().backward()
    # weights within 2e-6 relative, products of H terms within H * 2^-24 of their absolute sum
    mag = (rows.abs() * dout.cpu().double().abs()[:, None]).sum(2)
    part = w.detach() * (mag + (w.detach() * mag).sum(1, keepdim=True))
    bound = torch.zeros_like(z).scatter_(1, idx.cpu().long(), part * (4 * 2e-6 + H * 2.0 ** -24))
    ref.check(dlogits, z.grad, bound.detach())
    gone = (kept < 0).cpu()
    assert gone.any() and (dlogits.cpu().gather(1, idx.cpu().long())[gone] != 0).any()
