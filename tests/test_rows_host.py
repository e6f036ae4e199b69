"""Row operators without a GPU: what the calls refuse before anything is launched, and the 64-bit
forms' gradients against differences of their forward forms."""
import ctypes

import pytest
import torch

import rows_ref as ref

q = pytest.importorskip("quantized_mixture_experts_grouped_b200")

P = ctypes.c_void_p(4096)
P2 = ctypes.c_void_p(8192)
P3 = ctypes.c_void_p(1 << 20)
N = None
BF16, F16, F32 = q.MOE_DTYPE_BF16, q.MOE_DTYPE_F16, q.MOE_DTYPE_F32
ARG, SHAPE = q.MOE_ERR_ARG, q.MOE_ERR_SHAPE


def test_constants_match_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(root, "include", "moe_w4a16.h")).read(), flags=re.S)
    values = {n: int(v, 0) for n, v in re.findall(r"\b(MOE_[A-Z0-9_]+)\s*=\s*(0x[0-9a-fA-F]+|\d+)", text)}
    names = [n for n in values if n.startswith(("MOE_DTYPE_", "MOE_NORM_", "MOE_GATE_"))]
    assert len(names) == 9
    for n in names:
        assert values[n] == getattr(q, n), n


def dispatch(x=P, ldx=8, dt=BF16, idx=P, T=4, H=8, E=4, k=2, counts=P, offsets=P, perm=P, inv=P, xp=P2, ldp=8):
    return q.lib.moe_dispatch(x, ldx, dt, idx, T, H, E, k, counts, offsets, perm, inv, xp, ldp, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=N), ARG), (dict(idx=N), ARG), (dict(inv=N), ARG), (dict(xp=N), ARG), (dict(counts=N), ARG),
    (dict(T=-1), ARG), (dict(H=0), ARG), (dict(k=0), ARG), (dict(E=0), ARG), (dict(E=257), SHAPE),
    (dict(dt=3), ARG), (dict(dt=-1), ARG), (dict(ldx=-8), ARG), (dict(ldp=7), ARG), (dict(ldp=0), ARG),
    (dict(xp=P), ARG), (dict(T=1 << 30, k=4), SHAPE), (dict(H=(1 << 30) + 1, ldp=1 << 31), SHAPE),
    (dict(T=0, counts=N), ARG),
])
def test_dispatch_refusals(kw, code):
    assert dispatch(**kw) == code
    assert b"moe_dispatch" in q.lib.moe_last_error_string()


def test_dispatch_refuses_shared_index_buffers():
    """Each block reads every id while others write places: none may share a buffer."""
    ids = [ctypes.c_void_p(1 << i) for i in range(20, 26)]
    apart = dict(zip(("idx", "counts", "offsets", "perm", "inv", "xp"), ids))
    for name in ("counts", "offsets", "perm", "inv"):
        assert dispatch(**{**apart, name: apart["idx"]}) == ARG
        assert b"overlap" in q.lib.moe_last_error_string(), name
    assert dispatch(**{**apart, "perm": apart["inv"]}) == ARG


def test_combine_refusals():
    f = lambda yp=P, ldy=8, ydt=F32, inv=P, w=P, T=4, H=8, k=2, out=P2, ldo=8, odt=BF16: q.lib.moe_combine(
        yp, ldy, ydt, inv, w, T, H, k, out, ldo, odt, None)
    for kw in (dict(yp=N), dict(w=N), dict(out=N), dict(out=P), dict(ldo=7), dict(ldy=-1), dict(ydt=BF16, odt=F32),
               dict(ydt=BF16, odt=F16), dict(odt=9), dict(k=0), dict(H=0), dict(T=-2)):
        assert f(**kw) == ARG, kw
    assert f(T=1 << 30, k=2) == SHAPE
    assert f(T=0, yp=N, inv=N, w=N, out=N) == q.MOE_OK


def test_backward_refusals():
    f = lambda d=P, ldd=8, ddt=BF16, yp=P2, ldy=8, ydt=BF16, inv=P, w=P, T=4, H=8, k=2, dyp=P3, lddy=8, dw=P: \
        q.lib.moe_combine_backward(d, ldd, ddt, yp, ldy, ydt, inv, w, T, H, k, dyp, lddy, dw, None)
    for kw in (dict(d=N), dict(yp=N), dict(dyp=N, dw=N), dict(dyp=P2), dict(dyp=P), dict(lddy=4), dict(ydt=F16),
               dict(inv=N), dict(w=N), dict(ddt=7)):
        assert f(**kw) == ARG, kw
    g = lambda dxp=P, ld=8, dt=F16, inv=P, T=4, H=8, k=2, dx=P2, ldx=8: q.lib.moe_dispatch_backward(
        dxp, ld, dt, inv, T, H, k, dx, ldx, None)
    for kw in (dict(dxp=N), dict(dx=P), dict(dt=5), dict(ldx=3)):
        assert g(**kw) == ARG, kw
    h = lambda idx=P, w=P, d=P, T=4, E=8, k=2, out=P2, ld=8, dt=F32: q.lib.moe_route_topk_backward(
        idx, w, d, T, E, k, out, ld, dt, None)
    for kw, code in ((dict(idx=N), ARG), (dict(d=N), ARG), (dict(k=9), ARG), (dict(E=300, ld=300), SHAPE),
                     (dict(ld=7), ARG), (dict(dt=4), ARG), (dict(T=-1), ARG)):
        assert h(**kw) == code, kw
    assert h(T=0, idx=N, w=N, d=N, out=N) == q.MOE_OK


def test_norm_refusals():
    f = lambda h=P, ldh=8, dt=BF16, w=P, eps=1e-5, T=4, H=8, x=P2, ldx=8: q.lib.moe_norm_pre(
        h, ldh, dt, w, eps, T, H, x, ldx, None)
    for kw, code in ((dict(h=N), ARG), (dict(x=N), ARG), (dict(x=P), ARG), (dict(eps=0.0), ARG),
                     (dict(eps=float("nan")), ARG), (dict(eps=float("inf")), ARG), (dict(eps=-1.0), ARG),
                     (dict(H=16385, ldh=16385, ldx=16385), SHAPE), (dict(H=0), ARG), (dict(dt=3), ARG),
                     (dict(ldx=4), ARG), (dict(T=-1), ARG)):
        assert f(**kw) == code, kw
    g = lambda dx=P, h=P2, w=P, T=4, H=8, dres=N, ldr=0, dh=P3, ldd=8, dw=N, ws=N, wb=0: q.lib.moe_norm_pre_backward(
        dx, 8, h, 8, BF16, w, 1e-5, T, H, dres, ldr, dh, ldd, dw, ws, wb, None)
    for kw in (dict(dx=N), dict(dh=N), dict(dh=P), dict(dh=P2), dict(dres=P3, ldr=16), dict(dw=P), dict(ldd=2),
               dict(dw=P, ws=P, wb=16), dict(dw=P, ws=ctypes.c_void_p(4097), wb=1 << 30)):
        assert g(**kw) == ARG, kw
    with pytest.raises(q.MoeError):
        q.moe_norm_workspace_bytes(4, 20000)
    assert q.moe_norm_workspace_bytes(0, 8) > 0
    # the size covers every smaller batch
    assert q.moe_norm_workspace_bytes(5, 64) <= q.moe_norm_workspace_bytes(5000, 64)


def test_post_refusals():
    def f(y=P, h=P2, w=N, gate=N, ldg=8, mode=0, eps=1e-5, T=4, H=8, flags=1, ho=P3, ldho=8, wn=N, xn=N, ldx=8):
        return q.lib.moe_norm_post(y, 8, h, 8, BF16, w, gate, ldg, mode, 1.0, eps, T, H, flags, ho, ldho, wn, xn, ldx,
                                   None)
    for kw in (dict(y=N), dict(h=N), dict(ho=N), dict(flags=4), dict(flags=3), dict(mode=1), dict(mode=5),
               dict(gate=P, mode=0), dict(ho=P), dict(ho=P2, ldho=16), dict(flags=3, xn=P3), dict(flags=3, xn=P),
               dict(flags=3, xn=P2), dict(ldho=7), dict(gate=P, mode=3, ldg=-1)):
        assert f(**kw) == ARG, kw
    assert f(H=20000, ldho=20000) == SHAPE

    def c(k=2, ydt=BF16, dt=BF16, inv=P, w=P, yo=N, ldyo=8, T=4):
        return q.lib.moe_combine_norm_post(P, 8, ydt, inv, w, k, P2, 8, dt, N, N, 0, 0, 1.0, 1e-5, T, 8, 1, P3, 8,
                                           N, N, 0, yo, ldyo, None)
    for kw in (dict(k=0), dict(ydt=F16), dict(ydt=BF16, dt=F32), dict(inv=N), dict(w=N), dict(yo=P), dict(yo=P2),
               dict(yo=P3), dict(yo=ctypes.c_void_p(1 << 21), ldyo=4)):
        assert c(**kw) == ARG, kw
    assert c(T=1 << 30, k=2) == SHAPE

    D, Y, HO, DX, DH, DY = (ctypes.c_void_p(1 << i) for i in range(20, 26))

    def b(dho=D, y=Y, gate=N, mode=0, flags=3, ho=HO, dx=DX, dh=DH, lddh=8, dy=DY, dw=N, dg=N, dwn=N, ws=N, wb=0):
        return q.lib.moe_norm_post_backward(dho, 8, y, 8, BF16, N, gate, 8, mode, 1.0, 1e-5, 4, 8, flags, ho, 8, N, dx,
                                            8, dh, lddh, dy, 8, dw, dg, 8, dwn, ws, wb, None)
    for kw in (dict(dho=N), dict(y=N), dict(dh=N), dict(dy=N), dict(ho=N), dict(dx=N), dict(flags=8),
               dict(flags=2, dw=P), dict(flags=1, dwn=P), dict(dg=P), dict(dh=Y), dict(dh=DY), dict(dy=D),
               dict(dh=HO), dict(dy=DX), dict(dh=D, lddh=16), dict(gate=P, mode=3, dg=DH), dict(mode=2),
               dict(dw=P), dict(gate=P, mode=1, dg=P2), dict(dw=P, ws=P, wb=8)):
        assert b(**kw) == ARG, kw


def test_binding_refuses_before_the_library():
    """Tensors on the CPU, wrong shapes and types: MoeError with the argument named."""
    x = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: q.moe_norm_pre(x, None, 1e-5, x),
                 lambda: q.moe_norm_pre(x.view(-1), None, 1e-5, x),
                 lambda: q.moe_dispatch(x, i, 4, i, i, i, i, x),
                 lambda: q.moe_dispatch(x, i.long(), 4, i, i, i, i, x),
                 lambda: q.moe_combine(x, i, x, x),
                 lambda: q.moe_norm_post(x, x, x, 1e-5, norm_y=False, w=x),
                 lambda: q.moe_norm_post(x, x, x, 1e-5, w_next=x),
                 lambda: q.moe_route_topk_backward(i, x, x, x)):
        with pytest.raises(q.MoeError) as ei:
            call()
        assert ei.value.code == ARG


# ------------------------------------------------------------------ the formulas' gradients

def _directional(f, args, grads, g):
    """The gradients of sum(c * f) against central differences of f along random directions, 64 bits.
    Differences of step s are off by O(s^2) of the third derivative and by 2^-53 * |f| / s: with
    s = 1e-5 about 1e-10 either way; 1e-6 of the largest term leaves room."""
    outs = f(*args)
    cs = [torch.randn(o.shape, generator=g, dtype=torch.float64) for o in outs]
    an = grads(cs)
    for i, a in enumerate(args):
        v = torch.randn(a.shape, generator=g, dtype=torch.float64)
        s = 1e-5
        up, dn = ([*args[:i], a + e * v, *args[i + 1:]] for e in (s, -s))
        num = sum((c * (o1 - o0)).sum() for c, o1, o0 in zip(cs, f(*up), f(*dn))) / (2 * s)
        want = (an[i] * v).sum()
        scale = float((an[i].abs() * v.abs()).sum())
        assert abs(float(num - want)) <= 1e-6 * scale, (i, float(num), float(want))


@pytest.mark.parametrize("norm_y", [True, False])
@pytest.mark.parametrize("gshape", [None, (12,), (5, 1), (5, 12)])
def test_norm_formulas_against_differences(norm_y, gshape):
    g = torch.Generator().manual_seed(1)
    T, H, eps, alpha = 5, 12, 1e-3, 0.7
    rnd = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)
    args = [rnd(T, H), rnd(T, H), rnd(H)] + ([rnd(*gshape)] if gshape else []) + ([rnd(H)] if norm_y else [])

    def split(a):
        return a[0], a[1], a[2], a[3] if gshape else None, a[-1] if norm_y else None

    def f(*a):
        y, h, wn, gate, w = split(a)
        ho, _, xn, _ = ref.norm_post(y, h, eps, alpha, norm_y, w, gate, wn, True)
        return ho, xn

    def grads(cs):
        y, h, wn, gate, w = split(args)
        ho = f(*args)[0]
        b = ref.norm_post_backward(cs[0], y, eps, alpha, norm_y, w, gate, ho, wn, cs[1])
        return [b["dy"][0], b["dh"][0], b["dw_next"][0]] + ([b["dgate"][0]] if gshape else []) + \
            ([b["dw"][0]] if norm_y else [])
    _directional(f, args, grads, g)


def test_row_formulas_against_differences():
    g = torch.Generator().manual_seed(2)
    T, k, H, E = 6, 3, 7, 5
    idx = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    idx[2] = -1
    idx[4, 1] = -1
    inv = ref.sort(idx, E)[3]
    yp = torch.randn(T * k, H, generator=g, dtype=torch.float64)
    wts = torch.randn(T, k, generator=g, dtype=torch.float64)

    def grads(cs):
        dyp, _, dw, _ = ref.combine_backward(cs[0], yp, inv, wts)
        return [torch.nan_to_num(dyp), dw]
    _directional(lambda y, w: [ref.combine(y, inv, w)[0]], [yp, wts], grads, g)
    # the router: weights renormalised over the chosen, as a function of all logits
    logits = torch.randn(T, E, generator=g, dtype=torch.float64)
    top = logits.topk(k, dim=1).indices

    def weights(z):
        p = torch.softmax(z, dim=1).gather(1, top)
        return [p / p.sum(1, keepdim=True)]
    _directional(weights, [logits], lambda cs: [ref.router_backward(top, weights(logits)[0], cs[0], E)[0]], g)
