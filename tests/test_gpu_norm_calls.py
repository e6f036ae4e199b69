"""Calls of the norms around a block that their documentation allows beside the ordinary ones."""
import pytest
import torch

import rows_ref as ref
from test_gpu_norm import CASES, EPS, cpu, post_inputs, ws_for
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


def sums_over_tokens(T):
    """Longest chain of a sum over the tokens as it is taken now: a block's rows (at least min(T, 148)
    blocks, or one block of up to four rows), up to five blocks of a run one after another, and trees of at
    most 4 + 5 steps."""
    return max(-(-T // min(T, 148)), min(T, 4)) + 5 + 9


def on_device(got, want, arith, what):
    """ref.check where the tensors are."""
    assert got.shape == want.shape and torch.isfinite(got).all(), what
    want, arith = want.double(), arith.double()
    lim = arith + ref.stored(want.abs() + arith, got.dtype)
    off = (got.double() - want).abs()
    assert not (off > lim).any(), (what, float((off / lim.clamp(min=1e-300)).max()))


# (T, H, pad, types): several rows to every block of each form of the gradient: words and single values
# from the ring, words and single values of one and two chunks above it
MANY = [(3000, 512, 0, "bf16 f16 f32"), (3001, 264, 8, "bf16 f16 f32"), (2500, 264, 1, "bf16 f16 f32"),
        (700, 4096, 0, "bf16 f32"), (700, 1031, 0, "bf16 f32"), (700, 4095, 0, "f16"),
        (4, 1536, 0, "bf16 f32"), (2, 4096, 1, "f16"), (500, 5000, 0, "bf16 f32"),
        (500, 5000, 1, "bf16 f32"), (400, 12544, 0, "bf16 f32"), (400, 12543, 0, "f16")]


@pytest.mark.parametrize("norm_y,gate,nxt", CASES)
@pytest.mark.parametrize("T,H,pad,dt", [(T, H, pad, dt) for T, H, pad, types in MANY for dt in types.split()])
def test_post_of_many_rows(norm_y, gate, nxt, T, H, pad, dt, monkeypatch):
    """Every combination of norms and gate where a block takes several rows: rows read ahead, slots used
    again, sums carried from row to row. Without the vectors' gradients the rows are the same."""
    monkeypatch.setattr(ref, "column_chain", sums_over_tokens)
    g = torch.Generator().manual_seed(T + H)
    dt, alpha = DT[dt], 0.75
    y, h, w, gt, wn = post_inputs(T, H, dt, g, pad, norm_y, gate, nxt)
    ho, xn = room(T, H, dt, pad), room(T, H, dt, pad) if nxt else None
    q.moe_norm_post(y, h, ho, EPS, alpha=alpha, norm_y=norm_y, w=w, gate=gt, w_next=wn, x_next=xn)
    rh, bh, rx, bx = ref.norm_post(y, h, EPS, alpha, norm_y, w, gt, wn, nxt)
    on_device(ho, rh, bh, "h_out")
    if nxt:
        on_device(xn, rx, bx, "x_next")
    dho, dxn = rows(T, H, dt, g, pad), rows(T, H, dt, g, pad) if nxt else None
    dh, dy = room(T, H, dt, pad), room(T, H, dt, pad)
    fp32 = lambda *s: torch.full(s, KEEP, device="cuda")
    dg = {"none": lambda: None, "channel": lambda: fp32(H), "token": lambda: fp32(T, 1),
          "full": lambda: room(T, H, dt, pad)}[gate]()
    dw, dn = fp32(H) if norm_y else None, fp32(H) if nxt else None
    kw = dict(alpha=alpha, norm_y=norm_y, w=w, gate=gt, h_out=ho if nxt else None, w_next=wn, dx_next=dxn)
    q.moe_norm_post_backward(dho, y, dh, dy, EPS, dw=dw, dgate=dg, dw_next=dn, ws=ws_for(T, H), **kw)
    want = ref.norm_post_backward(dho, y, EPS, alpha, norm_y, w, gt, ho if nxt else None, wn, dxn)
    for n, got in dict(dh=dh, dy=dy, dw=dw, dgate=dg, dw_next=dn).items():
        if got is not None:
            on_device(got, *want[n], n)
    dy2 = room(T, H, dt, pad)
    q.moe_norm_post_backward(dho, y, dho, dy2, EPS, **kw)             # dh in place of dh_out
    assert torch.equal(dho, dh) and torch.equal(dy2, dy)


@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("T,H,pad,dt", [(T, H, pad, dt) for T, H, pad, types in MANY for dt in types.split()])
def test_pre_of_many_rows(res, T, H, pad, dt, monkeypatch):
    monkeypatch.setattr(ref, "column_chain", sums_over_tokens)
    g = torch.Generator().manual_seed(T + H)
    dt = DT[dt]
    h, dx = rows(T, H, dt, g, pad), rows(T, H, dt, g, pad)
    w, dres = rows(1, H, dt, g)[0], rows(T, H, dt, g, pad) if res else None
    dh, d2, dw = room(T, H, dt, pad), room(T, H, dt, pad), torch.full((H,), KEEP, device="cuda")
    q.moe_norm_pre_backward(dx, h, w, EPS, dh, dres=dres, dw=dw, ws=ws_for(T, H))
    rh, bh, rw, bw = ref.norm_pre_backward(dx, h, w, EPS, dres)
    on_device(dh, rh, bh, "dh")
    on_device(dw, rw, bw, "dw")
    q.moe_norm_pre_backward(dx, h, w, EPS, d2, dres=dres)
    assert torch.equal(d2, dh)


@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
def test_no_tokens(gate):
    """An empty batch with every kind of gate and all gradients: vectors' gradients are zeros."""
    T, H, k, E = 0, 64, 2, 8
    e = lambda *s, dt=torch.bfloat16: torch.empty(s, dtype=dt, device="cuda")
    i32, f32 = torch.int32, torch.float32
    gt = {"none": None, "channel": torch.ones(H, dtype=torch.bfloat16, device="cuda"), "token": e(T, 1, dt=f32),
          "full": e(T, H)}[gate]
    dg = {"none": None, "channel": torch.ones(H, device="cuda"), "token": e(T, dt=f32), "full": e(T, H)}[gate]
    dw, dn = torch.ones(H, device="cuda"), torch.ones(H, device="cuda")
    q.moe_norm_post(e(T, H), e(T, H), e(T, H), EPS, gate=gt, x_next=e(T, H))
    q.moe_combine_norm_post(e(T * k, H), e(T, k, dt=i32), e(T, k, dt=f32), e(T, H), e(T, H), EPS, gate=gt,
                            x_next=e(T, H), y_out=e(T, H))
    q.moe_norm_post_backward(e(T, H), e(T, H), e(T, H), e(T, H), EPS, dw=dw, gate=gt, dgate=dg, h_out=e(T, H),
                             dx_next=e(T, H), dw_next=dn)
    assert (dw == 0).all() and (dn == 0).all() and (gate != "channel" or (dg == 0).all())
    q.moe_combine(e(T * k, H), e(T, k, dt=i32), e(T, k, dt=f32), e(T, H))
    q.moe_combine_backward(e(T, H), e(T * k, H), e(T, k, dt=i32), e(T, k, dt=f32), e(T * k, H), e(T, k, dt=f32))
    q.moe_dispatch_backward(e(T * k, H), e(T, k, dt=i32), e(T, H))
    q.moe_route_topk_backward(e(T, k, dt=i32), e(T, k, dt=f32), e(T, k, dt=f32), e(T, E))
