"""Calls of the norms around a block that their documentation allows beside the ordinary ones."""
import pytest
import torch

import rows_ref as ref
from test_gpu_norm import EPS, cpu, ws_for
from test_gpu_rows import DT, KEEP, room, routing, rows

pytestmark = pytest.mark.gpu

q = pytest.importorskip("quantized_mixture_experts_grouped_b200")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,pad", [(1, 8, 0), (5, 40, 0), (40, 40, 0), (300, 264, 8), (9, 31, 1)])
def test_gate_per_token_in_one_dimension(dt, T, H, pad):
    """One value per token as [T] is [T][1]: the same bits, forward and back. Where it could as well be
    the channels' gate (fp32 rows, T = H) it is that one, as before."""
    g = torch.Generator().manual_seed(T)
    dt = DT[dt]
    y, h, dho = (rows(T, H, dt, g, pad) for _ in range(3))
    E, k = 4, 2
    idx, wts = routing(T, E, k, g)
    inv, yp = ref.sort(idx, E)[3].cuda(), rows(T * k, H, dt, g, pad)
    flat = torch.rand(T, generator=g).cuda()
    wide = flat if dt == torch.float32 and T == H else flat[:, None]

    def run(gate, dgate):
        ho, hf, dh, dy = (room(T, H, dt, pad) for _ in range(4))
        q.moe_norm_post(y, h, ho, EPS, gate=gate)
        q.moe_combine_norm_post(yp, inv, wts.cuda(), h, hf, EPS, gate=gate)
        q.moe_norm_post_backward(dho, y, dh, dy, EPS, gate=gate, dgate=dgate, ws=ws_for(T, H))
        return ho, hf, dh, dy, dgate.reshape(-1)
    got = run(flat, torch.full((T,), KEEP, device="cuda"))
    want = run(wide, torch.full(wide.shape, KEEP, device="cuda"))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    if wide.dim() == 2:       # the gradient may have either form
        for gate, shape in ((flat, (T, 1)), (wide, (T,))):
            mixed = run(gate, torch.full(shape, KEEP, device="cuda"))
            for a, b in zip(mixed, want):
                assert torch.equal(a, b)
    rh = ref.norm_post(y.cpu(), h.cpu(), EPS, 1.0, True, None, cpu(wide), None, False)
    ref.check(got[0], *rh[:2], "h_out")
    for bad in (torch.rand(T + 1, device="cuda"), flat.double()):
        if bad.numel() != H:
            with pytest.raises(q.MoeError) as ei:
                q.moe_norm_post(y, h, room(T, H, dt, pad), EPS, gate=bad)
            assert ei.value.code == q.MOE_ERR_ARG
