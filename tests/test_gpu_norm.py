"""The norms before and after a block with its gate and scaled residual, and their gradients, on the
GPU against plain 64-bit forms (rows_ref) within the bounds derived there; and the whole block:
norm, router, sort, experts, way back, norm, and the gradients back to its inputs."""
import pytest
import torch

import rows_ref as ref
from test_gpu_rows import DT, KEEP, room, routing, rows

pytestmark = pytest.mark.gpu

q = pytest.importorskip("quantized_mixture_experts_grouped_b200")

EPS = 1e-5


def vec(H, dtype, g, mean=1.0, scale=0.2):
    return (torch.randn(H, generator=g) * scale + mean).to(dtype).cuda()


def make_gate(kind, T, H, dtype, g, pad):
    if kind == "none":
        return None
    if kind == "channel":
        return vec(H, dtype, g, 0.5)
    if kind == "token":
        return torch.rand((T, 1), generator=g).cuda()
    return rows(T, H, dtype, g, pad, 0.5)


def cpu(t):
    return None if t is None else t.cpu()


def ws_for(T, H):
    return torch.full((q.moe_norm_workspace_bytes(T, H),), 0x7f, dtype=torch.uint8, device="cuda")


# one value; odd widths (single values); one, several and all warps; two chunks per thread
WIDTHS = [(1, 1), (3, 7), (2, 2048), (5, 1031), (4, 4096), (3, 8192), (2, 12288 + 256), (2, 16384), (1, 9001)]


# more tokens than blocks at each width, so that a block takes several rows
LONG = [(5000, 264), (3000, 512), (2500, 72), (1300, 2048), (700, 4096), (500, 8192),
        (70001, 8)]


@pytest.mark.parametrize("T,H", WIDTHS + [(700, 264)] + LONG)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 8, 1])
def test_pre(T, H, dt, pad):
    g = torch.Generator().manual_seed(H)
    dt = DT[dt]
    h, dx, dres = (rows(T, H, dt, g, pad) for _ in range(3))
    w = vec(H, dt, g)
    ws = ws_for(T, H)
    for wi, res in ((w, dres), (None, None)):
        x, dh, dw = room(T, H, dt, pad), room(T, H, dt, pad), torch.empty(H, device="cuda")
        q.moe_norm_pre(h, wi, EPS, x)
        ref.check(x, *ref.norm_pre(h.cpu(), cpu(wi), EPS), "x")
        q.moe_norm_pre_backward(dx, h, wi, EPS, dh, dres=res, dw=dw, ws=ws)
        rh, bh, rw, bw = ref.norm_pre_backward(dx.cpu(), h.cpu(), cpu(wi), EPS, cpu(res))
        ref.check(dh, rh, bh, "dh")
        ref.check(dw, rw, bw, "dw")
        d2 = res.clone() if res is not None and pad == 0 else None
        if d2 is not None:                # dh in place of the residual's gradient, without dw
            q.moe_norm_pre_backward(dx, h, wi, EPS, d2, dres=d2)
            assert torch.equal(d2, dh)


CASES = [(ny, gt, nx) for ny in (True, False) for gt in ("none", "channel", "token", "full") for nx in (True, False)]


def post_inputs(T, H, dt, g, pad, norm_y, gate, nxt):
    y, h = rows(T, H, dt, g, pad, 0.3), rows(T, H, dt, g, pad)
    w = vec(H, dt, g) if norm_y else None
    wn = vec(H, dt, g) if nxt else None
    return y, h, w, make_gate(gate, T, H, dt, g, pad), wn


def run_post_backward(T, H, dt, g, pad, y, h_out, w, gate, wn, norm_y, nxt, alpha, ws=None):
    """Runs and checks moe_norm_post_backward; returns its outputs."""
    dho = rows(T, H, dt, g, pad)
    dxn = rows(T, H, dt, g, pad) if nxt else None
    dh, dy = room(T, H, dt, pad), room(T, H, dt, pad)
    dw = torch.empty(H, device="cuda") if norm_y else None
    dwn = torch.empty(H, device="cuda") if nxt else None
    if gate is None:
        dg = None
    elif gate.dim() == 1:
        dg = torch.empty(H, device="cuda")
    elif gate.shape[1] == 1 and gate.dtype == torch.float32:
        dg = torch.empty((T, 1), device="cuda")
    else:
        dg = room(T, H, dt, pad)
    ws = ws_for(T, H) if ws is None else ws
    kw = dict(alpha=alpha, norm_y=norm_y, w=w, gate=gate, h_out=h_out if nxt else None, w_next=wn, dx_next=dxn)
    q.moe_norm_post_backward(dho, y, dh, dy, EPS, dw=dw, dgate=dg, dw_next=dwn, ws=ws, **kw)
    want = ref.norm_post_backward(dho.cpu(), y.cpu(), EPS, alpha, norm_y, cpu(w), cpu(gate), cpu(h_out), cpu(wn),
                                  cpu(dxn))
    got = dict(dh=dh, dy=dy, dw=dw, dgate=dg, dw_next=dwn)
    for n, v in got.items():
        if v is not None:
            ref.check(v, *want[n], n)
    # without the vectors' gradients: no workspace, the same rows; dh in place of dh_out
    dy2, dh2 = room(T, H, dt, pad), dho
    q.moe_norm_post_backward(dho, y, dh2, dy2, EPS, **kw)
    assert torch.equal(dy2, dy) and torch.equal(dh2, dh)
    return got


@pytest.mark.parametrize("norm_y,gate,nxt", CASES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,H,pad", [(1, 2048, 0), (5, 1031, 3), (9, 520, 8)])
def test_post(norm_y, gate, nxt, dt, T, H, pad):
    g = torch.Generator().manual_seed(T + H)
    dt = DT[dt]
    alpha = 0.75
    y, h, w, gt, wn = post_inputs(T, H, dt, g, pad, norm_y, gate, nxt)
    ho, xn = room(T, H, dt, pad), room(T, H, dt, pad) if nxt else None
    q.moe_norm_post(y, h, ho, EPS, alpha=alpha, norm_y=norm_y, w=w, gate=gt, w_next=wn, x_next=xn)
    rh, bh, rx, bx = ref.norm_post(y.cpu(), h.cpu(), EPS, alpha, norm_y, cpu(w), cpu(gt), cpu(wn), nxt)
    ref.check(ho, rh, bh, "h_out")
    if nxt:
        ref.check(xn, rx, bx, "x_next")
    run_post_backward(T, H, dt, g, pad, y, ho, w, gt, wn, norm_y, nxt, alpha)
    # the residual stream in place
    q.moe_norm_post(y, h, h, EPS, alpha=alpha, norm_y=norm_y, w=w, gate=gt, w_next=wn, x_next=xn)
    assert torch.equal(h, ho)


@pytest.mark.parametrize("T,H", WIDTHS + [(700, 264), (1300, 72)] + LONG)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_post_widths(T, H, dt):
    """Every block size, more tokens than blocks (partial sums), no weights (ones)."""
    g = torch.Generator().manual_seed(H)
    dt = DT[dt]
    y, h, w, gt, wn = post_inputs(T, H, dt, g, 0, True, "channel", True)
    ho, xn = room(T, H, dt), room(T, H, dt)
    for wi, wni in ((w, wn), (None, None)):
        q.moe_norm_post(y, h, ho, EPS, w=wi, gate=gt, w_next=wni, x_next=xn)
        rh, bh, rx, bx = ref.norm_post(y.cpu(), h.cpu(), EPS, 1.0, True, cpu(wi), cpu(gt), cpu(wni), True)
        ref.check(ho, rh, bh, "h_out")
        ref.check(xn, rx, bx, "x_next")
        run_post_backward(T, H, dt, g, 0, y, ho, wi, gt, wni, True, True, 1.0)


@pytest.mark.parametrize("T,E,k,H", [(1, 64, 8, 2048), (16, 64, 8, 2048), (5, 7, 3, 1031), (6, 12, 9, 4096),
                                     (2, 8, 2, 16384), (300, 8, 2, 512), (280, 64, 8, 2048)])
@pytest.mark.parametrize("ydt,dt", [("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("norm_y,gate,nxt,drop,pad", [(True, "none", True, 0.0, 0), (True, "channel", True, 0.5, 8),
                                                       (False, "token", False, 0.5, 0), (False, "full", True, 0.0, 1)])
def test_fused_way_back(T, E, k, H, ydt, dt, norm_y, gate, nxt, drop, pad):
    g = torch.Generator().manual_seed(T + k)
    dt = DT[dt]
    idx, wts = routing(T, E, k, g, drop)
    if drop:
        idx[0] = -1                              # a token whose choices were all dropped: y = 0
    inv = ref.sort(idx, E)[3]
    yp = rows(T * k, H, DT[ydt], g, pad, 0.3)
    _, h, w, gt, wn = post_inputs(T, H, dt, g, pad, norm_y, gate, nxt)
    ho, xn, yo = room(T, H, dt, pad), room(T, H, dt, pad) if nxt else None, room(T, H, dt, pad)
    kw = dict(alpha=1.25, norm_y=norm_y, w=w, gate=gt, w_next=wn)
    q.moe_combine_norm_post(yp, inv.cuda(), wts.cuda(), h, ho, EPS, x_next=xn, y_out=yo, **kw)
    ry, by = ref.combine(yp.cpu(), inv, wts)
    ref.check(yo, ry, by, "y")
    rh, bh, rx, bx = ref.norm_post(ry, h.cpu(), EPS, 1.25, norm_y, cpu(w), cpu(gt), cpu(wn), nxt, y_err=by)
    ref.check(ho, rh, bh, "h_out")
    if nxt:
        ref.check(xn, rx, bx, "x_next")
    h2 = h.clone() if pad == 0 else None          # in place, y not kept: the same bits
    if h2 is not None:
        x2 = torch.empty_like(xn) if nxt else None
        q.moe_combine_norm_post(yp, inv.cuda(), wts.cuda(), h2, h2, EPS, x_next=x2, **kw)
        assert torch.equal(h2, ho) and (not nxt or torch.equal(x2, xn))


def test_rows_of_zeros_and_no_rows():
    """A row of zeros norms to zeros with finite gradients; no rows at all: sums are zeros."""
    H = 256
    z = torch.zeros((3, H), device="cuda")
    x, dh, dw = torch.empty_like(z), torch.empty_like(z), torch.empty(H, device="cuda")
    ws = ws_for(3, H)
    q.moe_norm_pre(z, None, EPS, x)
    assert (x == 0).all()
    one = torch.ones_like(z)
    q.moe_norm_pre_backward(one, z, None, EPS, dh, dw=dw, ws=ws)
    r, b, rw, bw = ref.norm_pre_backward(one.cpu(), z.cpu(), None, EPS, None)
    ref.check(dh, r, b)
    ref.check(dw, rw, bw)
    e = torch.empty((0, H), device="cuda")
    dw.fill_(KEEP)
    dg = torch.full((H,), KEEP, device="cuda")
    dn = torch.full((H,), KEEP, device="cuda")
    q.moe_norm_pre(e, None, EPS, e.clone())
    q.moe_norm_post(e, e.clone(), e.clone(), EPS)
    q.moe_norm_post_backward(e, e.clone(), e.clone(), e.clone(), EPS, dw=dw, gate=torch.ones(H, device="cuda"),
                             dgate=dg, h_out=e.clone(), dx_next=e.clone(), dw_next=dn)
    assert (dw == 0).all() and (dg == 0).all() and (dn == 0).all()


def test_infinities_stay_in_their_row():
    H = 512
    g = torch.Generator().manual_seed(3)
    y, h = rows(3, H, torch.bfloat16, g), rows(3, H, torch.bfloat16, g)
    want, xw = torch.empty_like(h), torch.empty_like(h)
    q.moe_norm_post(y, h, want, EPS, x_next=xw)
    y2 = y.clone()
    y2[1, 7] = float("inf")
    y2[1, 9] = float("nan")
    got, xg = torch.empty_like(h), torch.empty_like(h)
    q.moe_norm_post(y2, h, got, EPS, x_next=xg)
    assert got[1].isnan().any() and xg[1].isnan().all()
    for r in (0, 2):
        assert torch.equal(got[r], want[r]) and torch.equal(xg[r], xw[r])


def test_large_values_and_small():
    """Mean squares near both ends of what fp32 sums hold."""
    g = torch.Generator().manual_seed(5)
    for s in (1e15, 1e-12):
        h, dx = rows(4, 1024, torch.float32, g, 0, s), rows(4, 1024, torch.float32, g)
        x, dh = torch.empty_like(h), torch.empty_like(h)
        q.moe_norm_pre(h, None, EPS, x)
        ref.check(x, *ref.norm_pre(h.cpu(), None, EPS), "x")
        q.moe_norm_pre_backward(dx, h, None, EPS, dh)
        r, b, _, _ = ref.norm_pre_backward(dx.cpu(), h.cpu(), None, EPS, None)
        ref.check(dh, r, b, "dh")


def test_fused_equals_its_parts():
    """x_next of moe_norm_post is the norm of the residual before its rounding: in fp32, where
    nothing is rounded in between, the same bits as moe_norm_pre on h_out."""
    g = torch.Generator().manual_seed(6)
    T, H = 37, 2048
    y, h, w, gt, wn = post_inputs(T, H, torch.float32, g, 0, True, "channel", True)
    ho, xn, x2 = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    q.moe_norm_post(y, h, ho, EPS, w=w, gate=gt, w_next=wn, x_next=xn)
    q.moe_norm_pre(ho, wn, EPS, x2)
    assert torch.equal(xn, x2)


def test_two_graphs_share_a_workspace():
    """Two captured backward passes with one workspace, replayed in turn: each gives its own sums."""
    g = torch.Generator().manual_seed(7)
    T, H = 2000, 512
    ws = ws_for(T, H)
    sets = []
    for _ in range(2):
        dx, h = rows(T, H, torch.bfloat16, g), rows(T, H, torch.bfloat16, g)
        dh, dw = torch.empty_like(h), torch.empty(H, device="cuda")
        q.moe_norm_pre_backward(dx, h, None, EPS, dh, dw=dw, ws=ws)
        torch.cuda.synchronize()
        want = (dh.clone(), dw.clone())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q.moe_norm_pre_backward(dx, h, None, EPS, dh, dw=dw, ws=ws)
        sets.append((graph, dh, dw, want, dx, h))       # the graph reads dx and h: they stay
    for _, dh, dw, *_ in sets:
        dh.zero_()
        dw.zero_()
    for i in (0, 1, 0, 1, 1):
        sets[i][0].replay()
    torch.cuda.synchronize()
    for _, dh, dw, want, *_ in sets:
        assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])


@pytest.mark.parametrize("T,drop", [(1, False), (13, True), (300, True)])
def test_whole_block_against_autograd(T, drop):
    """Norm, router, sort, SwiGLU experts (torch, fp32 rows), fused way back with gate and residual,
    and every gradient, against torch's autograd in 64 bits. fp32 throughout; the experts' products
    in fp32 bring the only errors that rows_ref does not bound: 1e-4 of each result's norm covers
    sums of 256 products at 2^-24 each through five chained steps with room to spare."""
    torch.manual_seed(T)
    H, I, E, k, alpha = 256, 128, 8, 2, 0.9
    dev = "cuda"
    mk = lambda *s, m=0.0, f=1.0: (torch.randn(s, device=dev) * f + m)
    h, w, wp, wn, gate = mk(T, H), mk(H, m=1, f=.1), mk(H, m=1, f=.1), mk(H, m=1, f=.1), mk(H, m=.5, f=.1)
    wr = mk(E, H, f=H ** -0.5)
    w1, w2, w3 = mk(E, I, H, f=H ** -0.5), mk(E, I, H, f=H ** -0.5), mk(E, H, I, f=I ** -0.5)
    # forward, the library's calls
    x = torch.empty_like(h)
    q.moe_norm_pre(h, w, EPS, x)
    logits = x @ wr.T
    lb = logits.bfloat16()
    idx, wts = torch.empty((T, k), dtype=torch.int32, device=dev), torch.empty((T, k), device=dev)
    q.moe_route_topk(lb, k, idx, wts)
    if drop:
        idx[::3, 1] = -1
    i32 = dict(dtype=torch.int32, device=dev)
    counts, offsets, perm, inv = (torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32),
                                  torch.empty((T, k), **i32))
    xp = torch.zeros((T * k, H), device=dev)
    q.moe_dispatch(x, idx, E, counts, offsets, perm, inv, xp)
    off = offsets.tolist()
    xps = [xp[off[e]:off[e + 1]].detach().requires_grad_() for e in range(E)]
    ys = [(torch.nn.functional.silu(a @ w1[e].T) * (a @ w2[e].T)) @ w3[e].T for e, a in enumerate(xps)]
    yp = torch.zeros((T * k, H), device=dev)
    yp[:off[-1]] = torch.cat(ys).detach()
    ho, xn, y = torch.empty_like(h), torch.empty_like(h), torch.empty_like(h)
    q.moe_combine_norm_post(yp, inv, wts, h, ho, EPS, alpha=alpha, w=wp, gate=gate, w_next=wn, x_next=xn, y_out=y)
    # backward
    dho, dxn = mk(T, H), mk(T, H)
    ws = ws_for(T, H)
    dh, dy, dwp, dgate, dwn = (torch.empty_like(h), torch.empty_like(h), torch.empty(H, device=dev),
                               torch.empty(H, device=dev), torch.empty(H, device=dev))
    q.moe_norm_post_backward(dho, y, dh, dy, EPS, alpha=alpha, w=wp, dw=dwp, gate=gate, dgate=dgate, h_out=ho,
                             w_next=wn, dx_next=dxn, dw_next=dwn, ws=ws)
    dyp, dwts, dlog = torch.zeros_like(yp), torch.empty_like(wts), torch.empty((T, E), device=dev)
    q.moe_combine_backward(dy, yp, inv, wts, dyp, dwts)
    full = torch.where(idx < 0, lb.float().topk(k, 1).indices.int(), idx)    # the router's own choice
    q.moe_route_topk_backward(full, wts, dwts, dlog)
    torch.autograd.backward(ys, [dyp[off[e]:off[e + 1]] for e in range(E)])
    dxp = torch.zeros_like(xp)
    dxp[:off[-1]] = torch.cat([a.grad for a in xps])
    dx, dhin, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(H, device=dev)
    q.moe_dispatch_backward(dxp, inv, dx)
    dx += dlog @ wr
    q.moe_norm_pre_backward(dx, h, w, EPS, dhin, dres=dh, dw=dw, ws=ws)
    # the same in 64 bits
    D = lambda t: t.double().requires_grad_()
    h6, w6, wp6, wn6, g6 = D(h), D(w), D(wp), D(wn), D(gate)
    rms = lambda v: v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS)
    x6 = rms(h6) * w6
    z6 = x6 @ wr.double().T
    z6 = z6 + (lb.double() - z6).detach()               # the router read rounded logits
    w6t = torch.softmax(z6.gather(1, full.long()), 1)
    y6 = torch.zeros((T, H), device=dev, dtype=torch.float64)
    for j in range(k):
        for e in range(E):
            t = torch.nonzero(idx[:, j] == e)[:, 0]
            a = x6[t]
            o = (torch.nn.functional.silu(a @ w1[e].double().T) * (a @ w2[e].double().T)) @ w3[e].double().T
            y6 = y6.index_add(0, t, o * w6t[t, j, None])
    ho6 = alpha * h6 + g6 * (rms(y6) * wp6)
    xn6 = rms(ho6) * wn6
    torch.autograd.backward([ho6, xn6], [dho.double(), dxn.double()])
    for name, got, want in (("h_out", ho, ho6), ("x_next", xn, xn6), ("dh", dhin, h6.grad), ("dw", dw, w6.grad),
                            ("dw_post", dwp, wp6.grad), ("dw_next", dwn, wn6.grad), ("dgate", dgate, g6.grad)):
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 1e-4, (name, rel)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [512, 4096])
def test_vectors_on_any_boundary(dt, H):
    """Weights, gate and the vectors' gradients one element into their buffers; a misaligned gradient
    beside aligned weights."""
    g = torch.Generator().manual_seed(H)
    dt, T = DT[dt], 600
    y, h = rows(T, H, dt, g, 0, 0.3), rows(T, H, dt, g)
    odd = lambda m: (torch.randn(H + 1, generator=g) * 0.2 + m).to(dt).cuda()[1:]
    ho, xn = room(T, H, dt), room(T, H, dt)
    for vectors in ((odd(1), odd(0.5), odd(1)), tuple(vec(H, dt, g) for _ in range(3))):
        w, gate, wn = vectors
        q.moe_norm_post(y, h, ho, EPS, w=w, gate=gate, w_next=wn, x_next=xn)
        rh, bh, rx, bx = ref.norm_post(y.cpu(), h.cpu(), EPS, 1.0, True, w.cpu(), gate.cpu(), wn.cpu(), True)
        ref.check(ho, rh, bh, "h_out")
        ref.check(xn, rx, bx, "x_next")
        for n in (T, 1):                       # one row: written by the first launch itself
            dho, dxn, dh, dy = (rows(n, H, dt, g) for _ in range(4))
            dw, dg, dn = (torch.full((H + 1,), KEEP, device="cuda")[1:] for _ in range(3))
            q.moe_norm_post_backward(dho, y[:n], dh, dy, EPS, w=w, dw=dw, gate=gate, dgate=dg, h_out=ho[:n], w_next=wn,
                                     dx_next=dxn, dw_next=dn, ws=ws_for(n, H))
            want = ref.norm_post_backward(dho.cpu(), y[:n].cpu(), EPS, 1.0, True, w.cpu(), gate.cpu(), ho[:n].cpu(),
                                          wn.cpu(), dxn.cpu())
            for name, got in (("dh", dh), ("dy", dy), ("dw", dw), ("dgate", dg), ("dw_next", dn)):
                ref.check(got, *want[name], name)


def at(n, H, dt, off, g, ld=None, scale=1.0):
    """Rows [n][H] that start `off` values into their buffer, ld apart (0: one row for all)."""
    ld = H if ld is None else ld
    buf = (torch.randn(off + max(n - 1, 0) * ld + H, generator=g) * scale).to(dt).cuda()
    return torch.as_strided(buf, (n, H), (ld, 1), off)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("H", [1, 3, 136, 1000, 1031, 2050, 4095])
@pytest.mark.parametrize("T", [1, 2, 700])
def test_rows_that_start_anywhere(dt, H, T):
    """Every tensor at an offset of its own, contiguous and strided rows, inputs that repeat one row."""
    g = torch.Generator().manual_seed(H + T)
    dt = DT[dt]
    n = 0

    def new(ld=None, scale=1.0):
        nonlocal n
        n += 3
        return at(T, H, dt, n % 8, g, ld, scale)
    y, h, gate = new(scale=0.3), new(0), new(H + 3)
    w, wn = at(1, H, dt, 5, g)[0], at(1, H, dt, 2, g)[0]
    ho, xn = new(H + 1), new()
    q.moe_norm_post(y, h, ho, EPS, alpha=0.5, w=w, gate=gate, w_next=wn, x_next=xn)
    rh, bh, rx, bx = ref.norm_post(y.cpu(), h.cpu(), EPS, 0.5, True, w.cpu(), gate.cpu(), wn.cpu(), True)
    ref.check(ho, rh, bh, "h_out")
    ref.check(xn, rx, bx, "x_next")
    dho, dxn, dh, dy, dg = new(0), new(), new(H + 1), new(), new(H + 5)
    dw, dn = torch.empty(H, device="cuda"), torch.empty(H, device="cuda")
    ws = ws_for(T, H)
    q.moe_norm_post_backward(dho, y, dh, dy, EPS, alpha=0.5, w=w, dw=dw, gate=gate, dgate=dg, h_out=ho, w_next=wn,
                             dx_next=dxn, dw_next=dn, ws=ws)
    want = ref.norm_post_backward(dho.cpu(), y.cpu(), EPS, 0.5, True, w.cpu(), gate.cpu(), ho.cpu(), wn.cpu(),
                                  dxn.cpu())
    for name, got in (("dh", dh), ("dy", dy), ("dw", dw), ("dgate", dg), ("dw_next", dn)):
        ref.check(got, *want[name], name)
    x, dx, dhp, res = new(), new(0), new(), new()
    q.moe_norm_pre(y, w, EPS, x)
    ref.check(x, *ref.norm_pre(y.cpu(), w.cpu(), EPS), "x")
    q.moe_norm_pre_backward(dx, y, w, EPS, dhp, dres=res, dw=dw, ws=ws)
    r, b, rw, bw = ref.norm_pre_backward(dx.cpu(), y.cpu(), w.cpu(), EPS, res.cpu())
    ref.check(dhp, r, b, "dh pre")
    ref.check(dw, rw, bw, "dw pre")
    q.moe_norm_pre_backward(dx, y, w, EPS, res, dres=res)              # in place
    assert torch.equal(res, dhp)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("H", [3, 136, 1031])
@pytest.mark.parametrize("T,k", [(9, 3), (900, 4)])
def test_way_back_of_rows_that_start_anywhere(dt, H, T, k):
    g = torch.Generator().manual_seed(H)
    dt, E = DT[dt], 6
    idx, wts = routing(T, E, k, g, 0.2)
    x, xp = at(T, H, dt, 3, g), at(T * k, H, dt, 6, g, H + 1)
    before = xp.clone()
    i32 = dict(dtype=torch.int32, device="cuda")
    inv, w = torch.empty((T, k), **i32), wts.cuda()
    q.moe_dispatch(x, idx.cuda(), E, torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32), inv,
                   xp)
    perm = ref.sort(idx, E)[2]
    assert torch.equal(xp[:len(perm)], x[(perm // k).long().cuda()]) and torch.equal(xp[len(perm):], before[len(perm):])
    out, h, ho = at(T, H, dt, 1, g), at(T, H, dt, 7, g, 0), at(T, H, dt, 4, g)
    q.moe_combine(xp, inv, w, out)
    r, b = ref.combine(xp.cpu(), inv.cpu(), wts)
    ref.check(out, r, b, "out")
    q.moe_combine_norm_post(xp, inv, w, h, ho, EPS)
    rh, bh, _, _ = ref.norm_post(r, h.cpu(), EPS, 1.0, True, None, None, None, False, y_err=b)
    ref.check(ho, rh, bh, "h_out")
    if T < 100:
        dyp, dw = at(T * k, H, dt, 5, g), torch.empty((T, k), device="cuda")
        q.moe_combine_backward(h, xp, inv, w, dyp, dw)
        rd, bd, rw, bw = ref.combine_backward(h.cpu(), xp.cpu(), inv.cpu(), wts)
        live = ~rd.isnan().any(1)
        ref.check(dyp.cpu()[live], rd[live], bd[live], "dyp")
        ref.check(dw, rw, bw, "dwts")


@pytest.mark.parametrize("H,pad", [(2048, 0), (1031, 0), (512, 1), (4096, 8)])
def test_gradients_repeat(H, pad):
    """The same bits from twenty runs, with another kernel's work before each."""
    g = torch.Generator().manual_seed(H)
    T, dt = 3000, torch.bfloat16
    y, h, dho, dxn = (rows(T, H, dt, g, pad) for _ in range(4))
    w, wn, gate = (vec(H, dt, g) for _ in range(3))
    ws, first = ws_for(T, H), None
    for _ in range(20):
        dh, dy = room(T, H, dt, pad), room(T, H, dt, pad)
        sums = [torch.full((H,), KEEP, device="cuda") for _ in range(3)]
        ws.fill_(0xff)
        q.moe_norm_post_backward(dho, y, dh, dy, EPS, w=w, dw=sums[0], gate=gate, dgate=sums[1], h_out=h, w_next=wn,
                                 dx_next=dxn, dw_next=sums[2], ws=ws)
        got = [dh, dy, *sums]
        first = got if first is None else first
        for a, b in zip(got, first):
            assert torch.equal(a, b)
