"""Rows sorted by expert and back, their gradients and the router's, on the GPU against plain 64-bit
forms (rows_ref): integers and copied rows bit-exact, sums within the bounds derived there."""
import numpy as np
import pytest
import torch

import rows_ref as ref

pytestmark = pytest.mark.gpu

q = pytest.importorskip("quantized_mixture_experts_grouped_b200")

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
KEEP = 12345.0      # what buffers hold before a call: exact in every type


def rows(n, H, dtype, g, pad=0, scale=1.0):
    """Device rows [n][H] inside rows of H + pad, values drawn on the host."""
    b = (torch.randn((n, H + pad), generator=g) * scale).to(dtype)
    return b.cuda()[:, :H]


def room(n, H, dtype, pad=0):
    return torch.full((n, H + pad), KEEP, dtype=dtype, device="cuda")[:, :H]


def routing(T, E, k, g, drop=0.0, skew=False):
    z = torch.rand((T, E), generator=g)
    if skew:
        z = z - torch.linspace(0, 1.5, E)
    idx = z.argsort(dim=1, descending=True)[:, :k].int()
    if drop:
        idx[torch.rand((T, k), generator=g) < drop] = -1
        idx[torch.rand((T, k), generator=g) < drop / 4] = E          # past the last expert
    wts = torch.softmax(torch.randn((T, k), generator=g), dim=1)
    return idx.contiguous(), wts


def dispatch(x, idx, E, pad=0, stream=None):
    T, k = idx.shape
    i32 = dict(dtype=torch.int32, device="cuda")
    o = dict(counts=torch.full((E,), -7, **i32), offsets=torch.full((E + 1,), -7, **i32),
             perm=torch.full((T * k,), -7, **i32), inv=torch.full((T, k), -7, **i32),
             xp=room(T * k, x.shape[1], x.dtype, pad))
    q.moe_dispatch(x, idx.cuda(), E, o["counts"], o["offsets"], o["perm"], o["inv"], o["xp"], stream=stream)
    return o


def check_dispatch(o, x, idx, E):
    counts, offsets, perm, inv = ref.sort(idx, E)
    n, k = len(perm), idx.shape[1]
    torch.testing.assert_close(o["counts"].cpu(), counts, rtol=0, atol=0)
    torch.testing.assert_close(o["offsets"].cpu(), offsets, rtol=0, atol=0)
    torch.testing.assert_close(o["inv"].cpu(), inv, rtol=0, atol=0)
    torch.testing.assert_close(o["perm"].cpu()[:n], perm, rtol=0, atol=0)
    assert (o["perm"].cpu()[n:] == -7).all()
    xp = o["xp"]
    assert torch.equal(xp[:n], x[(perm // k).long().cuda()])
    assert (xp[n:] == KEEP).all()
    if xp.stride(0) > xp.shape[1] and xp.shape[0] > 1:      # the buffer between the rows
        whole = torch.as_strided(xp, (xp.shape[0], xp.stride(0)), (xp.stride(0), 1))
        assert (whole[:, xp.shape[1]:] == KEEP).all()


# (T, E, k, H): one token; one pair; odd widths; 2048 pairs (the one-launch form's last) and 2049;
# one round and many of the sort's warps; every expert chosen; k past a warp
SHAPES = [(1, 64, 8, 2048), (1, 1, 1, 1), (3, 5, 2, 7), (17, 7, 3, 1031), (256, 64, 8, 128), (683, 9, 3, 40),
          (2049, 256, 1, 24), (5000, 256, 2, 16), (33, 40, 40, 136), (9, 256, 256, 8)]


@pytest.mark.parametrize("T,E,k,H", SHAPES)
@pytest.mark.parametrize("drop", [0.0, 0.3])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_dispatch(T, E, k, H, drop, dt):
    g = torch.Generator().manual_seed(T + E)
    idx, _ = routing(T, E, k, g, drop)
    x = rows(T, H, DT[dt], g)
    check_dispatch(dispatch(x, idx, E), x, idx, E)


@pytest.mark.parametrize("pad_in,pad_out,H", [(8, 8, 64), (1, 0, 64), (0, 3, 64), (5, 5, 63), (4, 2, 64)])
@pytest.mark.parametrize("T", [21, 900])
def test_dispatch_strides(pad_in, pad_out, H, T):
    """Rows inside wider buffers, on and off 16-byte boundaries; what lies between them stays."""
    g = torch.Generator().manual_seed(3)
    idx, _ = routing(T, 8, 3, g, 0.2)
    for dt in DT.values():
        x = rows(T, H, dt, g, pad_in)
        check_dispatch(dispatch(x, idx, 8, pad_out), x, idx, 8)
    one = rows(1, H, torch.bfloat16, g).expand(T, H)          # one row for every token: stride 0
    check_dispatch(dispatch(one, idx, 8, pad_out), one, idx, 8)


def test_dispatch_extremes():
    g = torch.Generator().manual_seed(4)
    for T in (5, 1000):
        x = rows(T, 32, torch.bfloat16, g)
        for idx in (torch.full((T, 4), -1), torch.full((T, 4), 2), torch.full((T, 4), 3)):
            idx = idx.int()                                   # all dropped; all to one expert; to the last
            check_dispatch(dispatch(x, idx, 4), x, idx, 4)
    x = rows(0, 32, torch.bfloat16, g)                        # no tokens
    o = dispatch(x, torch.zeros((0, 4), dtype=torch.int32), 4)
    assert (o["counts"] == 0).all() and (o["offsets"] == 0).all()


def test_sort_of_a_long_batch():
    """131072 pairs, skewed: against torch's stable sort."""
    g = torch.Generator().manual_seed(5)
    T, E, k = 16384, 64, 8
    idx, _ = routing(T, E, k, g, 0.05, skew=True)
    x = rows(T, 8, torch.bfloat16, g)
    o = dispatch(x, idx, E)
    e = idx.reshape(-1).long()
    ok = (e >= 0) & (e < E)
    key = torch.where(ok, e, E)
    perm = torch.sort(key, stable=True).indices
    n = int(ok.sum())
    assert torch.equal(o["perm"].cpu()[:n].long(), perm[:n])
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(T * k)
    assert torch.equal(o["inv"].cpu().view(-1).long(), torch.where(ok, inv, -1))
    assert torch.equal(o["counts"].cpu().long(), torch.bincount(key, minlength=E + 1)[:E])
    assert torch.equal(o["xp"][:n].cpu(), x.cpu()[perm[:n] // k])


def test_dispatch_rows_past_32_bit_offsets():
    """Places whose element offsets pass 2^31 (and byte offsets 2^32)."""
    g = torch.Generator().manual_seed(6)
    T, k, E, H = 20, 2, 4, 64
    ld = 1 << 26
    if torch.cuda.mem_get_info()[0] < 16 * 2**30:
        pytest.skip("needs 5.4 GB of device memory")
    buf = torch.empty((T * k - 1) * ld + H, dtype=torch.bfloat16, device="cuda")
    xp = torch.as_strided(buf, (T * k, H), (ld, 1))
    assert (T * k - 1) * ld > 2**31
    idx, wts = routing(T, E, k, g)
    x = rows(T, H, torch.bfloat16, g)
    i32 = dict(dtype=torch.int32, device="cuda")
    inv = torch.empty((T, k), **i32)
    q.moe_dispatch(x, idx.cuda(), E, torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(T * k, **i32), inv,
                   xp)
    perm = ref.sort(idx, E)[2]
    assert torch.equal(xp, x[(perm // k).long().cuda()])
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    q.moe_combine(xp, inv, wts.cuda(), out)
    r, b = ref.combine(xp.cpu(), inv.cpu(), wts)
    ref.check(out, r, b, "combine")


TYPES = [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16"), ("f32", "f16")]


@pytest.mark.parametrize("T,E,k,H", [(1, 64, 8, 2048), (1, 1, 1, 1), (5, 7, 3, 1031), (40, 16, 4, 4096), (7, 12, 9, 136),
                                     (6, 40, 17, 520)])
@pytest.mark.parametrize("ydt,odt", TYPES)
@pytest.mark.parametrize("drop,pad", [(0.0, 0), (0.4, 0), (0.4, 8), (0.0, 1)])
def test_combine_and_gradients(T, E, k, H, ydt, odt, drop, pad):
    g = torch.Generator().manual_seed(T * 7 + k)
    ydt, odt = DT[ydt], DT[odt]
    idx, wts = routing(T, E, k, g, drop)
    if T > 3 and drop:
        idx[2] = -1                       # a token with no choice left
    inv = ref.sort(idx, E)[3]
    P = T * k
    yp, dout = rows(P, H, ydt, g, pad, 0.3), rows(T, H, odt, g, pad)
    out = room(T, H, odt, pad)
    iv, w = inv.cuda(), wts.cuda()
    q.moe_combine(yp, iv, w, out)
    ref.check(out, *ref.combine(yp.cpu(), inv, wts), "combine")
    if T > 3 and drop:
        assert (out[2] == 0).all()
    dyp, dwts = room(P, H, ydt, pad), torch.full((T, k), KEEP, device="cuda")
    q.moe_combine_backward(dout, yp, iv, w, dyp, dwts)
    rd, bd, rw, bw = ref.combine_backward(dout.cpu(), yp.cpu(), inv, wts)
    live = ~rd.isnan().any(1)
    ref.check(dyp.cpu()[live], rd[live], bd[live], "dyp")
    assert (dyp.cpu()[~live] == KEEP).all()
    ref.check(dwts, rw, bw, "dwts")
    assert (dwts.cpu()[inv < 0] == 0).all()
    # each gradient alone gives the same bits
    d2, w2 = room(P, H, ydt, pad), torch.empty_like(dwts)
    if ydt == odt:
        q.moe_combine_backward(dout, None, iv, w, dyp=d2)
        assert torch.equal(d2, dyp)
    q.moe_combine_backward(dout, yp, iv, w, dwts=w2)
    assert torch.equal(w2, dwts)
    if ydt == odt:
        dx = room(T, H, odt, pad)
        q.moe_dispatch_backward(yp, iv, dx)
        ref.check(dx, *ref.combine(yp.cpu(), inv, None), "dx")


@pytest.mark.parametrize("T,E,k,H,pad", [(300, 16, 5, 1031, 0), (300, 16, 8, 1024, 1), (700, 8, 2, 255, 0), (1100, 8, 1, 333, 3),
                                         (260, 16, 7, 512, 0), (600, 8, 2, 640, 8), (600, 8, 2, 1032, 0), (400, 8, 3, 504, 0),
                                         (1100, 4, 1, 64, 0), (140, 40, 33, 600, 0), (130, 9, 9, 65, 0)])
@pytest.mark.parametrize("ydt,odt", TYPES)
def test_gradients_of_many_pairs(T, E, k, H, pad, ydt, odt):
    """Groups of one, two and four choices, the last not full, words and single values, tokens with none."""
    test_combine_and_gradients(T, E, k, H, ydt, odt, 0.4, pad)


def test_combine_ignores_what_dropped_rows_hold():
    """Infinities and NaN in rows no pair points to, and weights of dropped choices, change nothing."""
    g = torch.Generator().manual_seed(9)
    T, k, E, H = 12, 4, 6, 256
    idx, wts = routing(T, E, k, g, 0.5)
    inv = ref.sort(idx, E)[3]
    n = int((inv >= 0).sum())
    yp = rows(T * k, H, torch.bfloat16, g)
    dout = rows(T, H, torch.bfloat16, g)
    want, bound = ref.combine(yp.cpu(), inv, wts)
    _, _, dw, bw = ref.combine_backward(dout.cpu(), yp.cpu(), inv, wts)
    yp[n:] = float("nan")
    yp[n] = float("inf")
    w = wts.clone()
    w[inv < 0] = float("nan")
    out = room(T, H, torch.bfloat16)
    q.moe_combine(yp, inv.cuda(), w.cuda(), out)
    ref.check(out, want, bound)
    dyp, dwts = room(T * k, H, torch.bfloat16), torch.empty((T, k), device="cuda")
    q.moe_combine_backward(dout, yp, inv.cuda(), w.cuda(), dyp, dwts)
    ref.check(dwts, dw, bw)
    assert torch.isfinite(dyp).all()
    # values past the places' range are dropped too
    far = inv.clone()
    far[inv < 0] = T * k + 5
    out2 = torch.empty_like(out)
    q.moe_combine(yp, far.cuda(), w.cuda(), out2)
    assert torch.equal(out, out2)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (9, 8, 2), (70, 256, 8), (13, 100, 33), (3, 256, 256)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad", [0, 3])
def test_router_gradient(T, E, k, dt, pad):
    g = torch.Generator().manual_seed(E + k)
    idx, wts = routing(T, E, k, g)
    dwts = torch.randn((T, k), generator=g)
    if k > 2:
        idx[0, 1] = idx[0, 0]             # an id twice: the two add up
        idx[-1, 2] = -1                   # an id dropped after the router
    out = room(T, E, DT[dt], pad)
    q.moe_route_topk_backward(idx.cuda(), wts.cuda(), dwts.cuda(), out)
    ref.check(out, *ref.router_backward(idx, wts, dwts, E), "dlogits")


def test_router_and_its_gradient_against_autograd():
    """moe_route_topk's weights differentiated by torch in 64 bits."""
    g = torch.Generator().manual_seed(11)
    T, E, k = 50, 64, 8
    logits = torch.randn((T, E), generator=g).bfloat16()
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    wts = torch.empty((T, k), device="cuda")
    q.moe_route_topk(logits.cuda(), k, idx, wts)
    dwts = torch.randn((T, k), generator=g)
    out = torch.empty((T, E), device="cuda")
    q.moe_route_topk_backward(idx, wts, dwts.cuda(), out)
    z = logits.double().requires_grad_()
    p = torch.softmax(z, 1).gather(1, idx.cpu().long())
    (p / p.sum(1, keepdim=True) * dwts.double()).sum().backward()
    # the router's weights are within 2e-6 relative of the exact ones
    mag = wts.cpu().double() * (dwts.abs().double() + (wts.cpu() * dwts.abs()).sum(1, keepdim=True).double())
    bound = torch.zeros_like(z).scatter_(1, idx.cpu().long(), mag) * 2 * 2e-6
    # autograd's own rounding: it sums over all 64 experts in 64 bits, so an expert not chosen gets
    # up to 64 * 2^-53 of the row's terms where the exact gradient is 0
    ref.check(out, z.grad, bound.detach() + 64 * 2.0 ** -53 * mag.sum(1, keepdim=True))


def test_repeat_and_streams():
    """The same bits again, and from a stream of the caller's."""
    g = torch.Generator().manual_seed(12)
    T, E, k, H = 300, 16, 4, 512
    idx, wts = routing(T, E, k, g, 0.1)
    x, yp = rows(T, H, torch.bfloat16, g), rows(T * k, H, torch.bfloat16, g)
    a = dispatch(x, idx, E)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    w = wts.cuda()
    with torch.cuda.stream(s):
        b = dispatch(x, idx, E)
        o1 = room(T, H, torch.bfloat16)
        q.moe_combine(yp, b["inv"], w, o1)
    s.synchronize()
    for n in a:
        assert torch.equal(a[n], b[n]), n
    o2 = room(T, H, torch.bfloat16)
    q.moe_combine(yp, a["inv"], w, o2, stream=torch.cuda.current_stream())
    assert torch.equal(o1, o2)


def test_captured_and_replayed():
    """Sort, way back and both gradients in a CUDA graph, replayed on other routings (a batch of the
    one-launch form and one of the two-launch form)."""
    for T in (64, 600):
        g = torch.Generator().manual_seed(13)
        E, k, H = 16, 4, 256
        x, yp = rows(T, H, torch.bfloat16, g), rows(T * k, H, torch.bfloat16, g)
        idx = torch.zeros((T, k), dtype=torch.int32, device="cuda")
        wts = torch.zeros((T, k), device="cuda")
        i32 = dict(dtype=torch.int32, device="cuda")
        o = dict(counts=torch.empty(E, **i32), offsets=torch.empty(E + 1, **i32), perm=torch.full((T * k,), -7, **i32),
                 inv=torch.empty((T, k), **i32), xp=room(T * k, H, torch.bfloat16))
        out, dyp = room(T, H, torch.bfloat16), room(T * k, H, torch.bfloat16)
        dw, dl, dx = torch.empty_like(wts), torch.empty((T, E), device="cuda"), room(T, H, torch.bfloat16)

        def step():
            q.moe_dispatch(x, idx, E, o["counts"], o["offsets"], o["perm"], o["inv"], o["xp"])
            q.moe_combine(yp, o["inv"], wts, out)
            q.moe_combine_backward(x, yp, o["inv"], wts, dyp, dw)
            q.moe_route_topk_backward(idx, wts, dw, dl)
            q.moe_dispatch_backward(dyp, o["inv"], dx)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for seed in (1, 2):
            h = torch.Generator().manual_seed(seed)
            i, w = routing(T, E, k, h)
            idx.copy_(i)
            wts.copy_(w)
            graph.replay()
            torch.cuda.synchronize()
            check_dispatch(o, x, i, E)
            inv = o["inv"].cpu()
            ref.check(out, *ref.combine(yp.cpu(), inv, w), "out")
            rd, bd, rw, bw = ref.combine_backward(x.cpu(), yp.cpu(), inv, w)
            ref.check(dyp, rd, bd, "dyp")
            ref.check(dw, rw, bw, "dwts")
            ref.check(dl, *ref.router_backward(i, w, dw.cpu(), E), "dlogits")
            ref.check(dx, *ref.combine(dyp.cpu(), inv, None), "dx")


def test_binding_refusals_on_device():
    x = torch.zeros((4, 8), device="cuda", dtype=torch.bfloat16)
    i = torch.zeros((4, 2), device="cuda", dtype=torch.int32)
    w = torch.zeros((4, 2), device="cuda")
    yp = torch.zeros((8, 8), device="cuda")
    bad = [lambda: q.moe_combine(yp.t(), i, w, x), lambda: q.moe_combine(yp[:7], i, w, x),
           lambda: q.moe_combine(yp.half(), i, w, x), lambda: q.moe_combine(yp, i, w.half(), x),
           lambda: q.moe_combine(yp, i.long(), w, x), lambda: q.moe_combine(yp, i, w.cpu(), x),
           lambda: q.moe_combine(yp[:, ::2], i, w, x[:, :4]),
           lambda: q.moe_combine(yp, i, w, torch.zeros((1, 8), device="cuda").expand(4, 8)),
           lambda: q.moe_combine_backward(x, None, i, w, dwts=w.clone()),
           lambda: q.moe_combine_backward(x, yp, i, w),
           lambda: q.moe_norm_post_backward(x, x, x, x.clone(), 1e-5)]
    for n, call in enumerate(bad):
        with pytest.raises(q.MoeError) as ei:
            call()
        assert ei.value.code == q.MOE_ERR_ARG, n


def test_first_call_of_a_process_is_captured():
    """A process whose first calls are captured into a graph: nothing of them needs a warm-up."""
    import os
    import subprocess
    import sys
    code = """
import torch, quantized_mixture_experts_grouped_b200 as q
T, k, E, H = 400, 8, 16, 512
x = torch.randn(T, H, device="cuda").bfloat16()
idx = torch.rand(T, E, device="cuda").argsort(1)[:, :k].int().contiguous()
w = torch.ones(T, k, device="cuda")
i = dict(dtype=torch.int32, device="cuda")
c, o, p, inv = torch.empty(E, **i), torch.empty(E + 1, **i), torch.empty(T * k, **i), torch.empty(T, k, **i)
xp, out, dh, dw = torch.empty(T * k, H, device="cuda").bfloat16(), x.clone(), x.clone(), torch.empty(H, device="cuda")
ws = torch.empty(q.moe_norm_workspace_bytes(T, H), dtype=torch.uint8, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    q.moe_dispatch(x, idx, E, c, o, p, inv, xp)
    q.moe_combine(xp, inv, w, out)
    q.moe_norm_pre_backward(out, x, None, 1e-5, dh, dw=dw, ws=ws)
g.replay()
torch.cuda.synchronize()
assert torch.equal(out, x * 8) and torch.isfinite(dh).all() and torch.isfinite(dw).all()
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_two_threads_at_once():
    """Two host threads with streams of their own, both sorting, combining and norming in a loop."""
    import threading
    jobs = []
    for s in range(2):
        g = torch.Generator().manual_seed(20 + s)
        T, E, k, H = 300 + 77 * s, 16, 4, 512
        idx, wts = routing(T, E, k, g, 0.1)
        jobs.append((rows(T, H, torch.bfloat16, g), idx, E, wts.cuda(), torch.cuda.Stream()))
    want = []
    for x, idx, E, w, _ in jobs:
        o = dispatch(x, idx, E)
        out = room(*x.shape, x.dtype)
        q.moe_combine(o["xp"], o["inv"], w, out)
        want.append((o["inv"].clone(), out))
    torch.cuda.synchronize()
    wrong = []

    def work(n):
        x, idx, E, w, s = jobs[n]
        with torch.cuda.stream(s):
            for _ in range(50):
                o = dispatch(x, idx, E)
                out = room(*x.shape, x.dtype)
                q.moe_combine(o["xp"], o["inv"], w, out)
                s.synchronize()
                if not (torch.equal(o["inv"], want[n][0]) and torch.equal(out, want[n][1])):
                    wrong.append(n)
    threads = [threading.Thread(target=work, args=(n,)) for n in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
