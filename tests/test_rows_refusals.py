"""Refusals of the row operators one at a time: every buffer of the unchanged call is its own, so that a
case can only be refused for what it changes, and the message has to say what that is. No case is launched
(there need be no GPU): all are refused before."""
import ctypes

import pytest

q = pytest.importorskip("quantized_mixture_experts_grouped_b200")

N = None
BF16, F16, F32 = q.MOE_DTYPE_BF16, q.MOE_DTYPE_F16, q.MOE_DTYPE_F32
ARG, SHAPE = q.MOE_ERR_ARG, q.MOE_ERR_SHAPE


def buffers(names):
    """A distinct, well aligned address for each name (never read)."""
    return {n: ctypes.c_void_p((i + 1) << 30) for i, n in enumerate(names.split())}


def refused(fn, order, base, change, code, says):
    """fn on base with `change` (a name given as the value stands for that buffer)."""
    args = {**base, **{k: base[v] if isinstance(v, str) else v for k, v in change.items()}}
    assert set(args) == set(order.split()), set(args) ^ set(order.split())
    rc = getattr(q.lib, fn)(*(args[n] for n in order.split()), None)
    text = q.lib.moe_last_error_string().decode()
    assert rc == code, (change, rc, text)
    assert fn in text and says in text, (change, text)


POST = ("y ldy h ldh dt w gate ldg mode alpha eps T H flags ho ldho wn xn ldx")
POST_BASE = dict(buffers("y h w gate ho wn xn"), ldy=8, ldh=8, dt=BF16, ldg=8, mode=3, alpha=1.0, eps=1e-5, T=4, H=8,
                 flags=3, ldho=8, ldx=8)


@pytest.mark.parametrize("change,says", [
    (dict(ho="y"), "overlap"), (dict(ho="h", ldho=16), "overlap"), (dict(xn="ho"), "overlap"),
    (dict(xn="h"), "overlap"), (dict(xn="y"), "overlap"),
    (dict(ho="w"), "weight"), (dict(ho="wn"), "weight"), (dict(xn="w"), "weight"), (dict(xn="wn"), "weight"),
    (dict(ho="gate", ldho=16), "gate"), (dict(xn="gate", ldx=16), "gate"),
    (dict(ho="gate", mode=1), "gate"), (dict(xn="gate", mode=2), "gate")])
def test_post_outputs_overlap(change, says):
    refused("moe_norm_post", POST, POST_BASE, change, ARG, says)


FUSED = "yp ldyp ydt inv wts k h ldh dt w gate ldg mode alpha eps T H flags ho ldho wn xn ldx yo ldyo"
FUSED_BASE = dict(buffers("yp inv wts h w gate ho wn xn yo"), ldyp=8, ydt=BF16, k=2, ldh=8, dt=BF16, ldg=8, mode=3,
                  alpha=1.0, eps=1e-5, T=4, H=8, flags=3, ldho=8, ldx=8, ldyo=8)


@pytest.mark.parametrize("other", ["yp", "h", "ho", "xn", "w", "gate", "wn"])
@pytest.mark.parametrize("mode", [1, 2, 3])
def test_fused_y_out_overlaps(other, mode):
    """y_out is written before the gate and the weights are read."""
    refused("moe_combine_norm_post", FUSED, FUSED_BASE, dict(yo=other, mode=mode), ARG, "y_out overlaps")


BACK = ("dho lddho y ldy dt w gate ldg mode alpha eps T H flags ho ldho wn dx lddx dh lddh dy lddy dw dg lddg dwn ws "
        "wb")
BACK_BASE = dict(buffers("dho y w gate ho wn dx dh dy dw dg dwn ws"), lddho=8, ldy=8, dt=F32, ldg=8, mode=3, alpha=1.0,
                 eps=1e-5, T=4, H=8, flags=3, ldho=8, lddx=8, lddh=8, lddy=8, lddg=8, wb=1 << 30)


@pytest.mark.parametrize("change,says", [
    (dict(dh="y"), "overlap"), (dict(dh="dy"), "overlap"), (dict(dy="dho"), "overlap"), (dict(dy="y"), "overlap"),
    (dict(dh="ho"), "overlap"), (dict(dh="dx"), "overlap"), (dict(dy="ho"), "overlap"), (dict(dy="dx"), "overlap"),
    (dict(dh="dho", lddh=16), "overlap"), (dict(dh="gate"), "overlap"), (dict(dy="gate"), "overlap"),
    (dict(dg="dh"), "overlap"), (dict(dg="gate"), "overlap"), (dict(dg="ho"), "overlap"),
    (dict(dh="w"), "weight"), (dict(dh="wn"), "weight"), (dict(dy="w"), "weight"), (dict(dy="wn"), "weight"),
    (dict(dh="gate", mode=1), "gate"), (dict(dy="gate", mode=2), "gate"), (dict(dg="w"), "weight"),
    (dict(dg="wn", mode=1), "weight"),
    (dict(dw="dwn"), "share"), (dict(dw="dg", mode=1), "share"), (dict(dwn="dg", mode=1), "share")])
def test_post_gradients_overlap(change, says):
    refused("moe_norm_post_backward", BACK, BACK_BASE, change, ARG, says)


PRE = "h ldh dt w eps T H x ldx"
PRE_BACK = "dx lddx h ldh dt w eps T H dres ldr dh lddh dw ws wb"


@pytest.mark.parametrize("other", ["h", "w"])
def test_pre_output_overlaps(other):
    base = dict(buffers("h w x"), ldh=8, dt=BF16, eps=1e-5, T=4, H=8, ldx=8)
    refused("moe_norm_pre", PRE, base, dict(x=other), ARG, "overlap")


@pytest.mark.parametrize("change", [dict(dh="dx"), dict(dh="h"), dict(dh="w"), dict(dh="dres", lddh=16)])
def test_pre_gradient_overlaps(change):
    base = dict(buffers("dx h w dres dh dw ws"), lddx=8, ldh=8, dt=BF16, eps=1e-5, T=4, H=8, ldr=8, lddh=8, wb=1 << 30)
    refused("moe_norm_pre_backward", PRE_BACK, base, change, ARG, "overlap")


DISPATCH = "x ldx dt idx T H E k counts offsets perm inv xp ldp"
DISPATCH_BASE = dict(buffers("x idx counts offsets perm inv xp"), ldx=8, dt=BF16, T=4, H=8, E=4, k=2, ldp=8)


@pytest.mark.parametrize("change,code,says", [
    *[({n: N}, ARG, "null pointer") for n in ("x", "idx", "counts", "offsets", "perm", "inv", "xp")],
    (dict(T=0, counts=N), ARG, "null pointer"), (dict(T=0, offsets=N), ARG, "null pointer"),
    (dict(T=-1), ARG, "bad sizes"), (dict(H=0), ARG, "bad sizes"), (dict(k=0), ARG, "bad sizes"),
    (dict(E=0), ARG, "E=0"), (dict(E=257), SHAPE, "E=257"), (dict(dt=3), ARG, "type 3"), (dict(dt=-1), ARG, "type -1"),
    (dict(ldx=-8), ARG, "row stride -8 of x "), (dict(ldp=7), ARG, "row stride 7 of xp"),
    (dict(ldp=0), ARG, "row stride 0 of xp"), (dict(xp="x"), ARG, "xp overlaps x"),
    (dict(T=1 << 30, k=4), SHAPE, "T*k"), (dict(H=(1 << 30) + 1, ldp=1 << 31), SHAPE, "2^30"),
    *[({n: "idx"}, ARG, "index outputs overlap") for n in ("counts", "offsets", "perm", "inv")],
    *[({a: b}, ARG, "index outputs overlap") for a, b in (("perm", "inv"), ("counts", "offsets"), ("counts", "perm"),
                                                           ("counts", "inv"), ("offsets", "perm"), ("offsets", "inv"))],
    (dict(T=0, counts="offsets"), ARG, "index outputs overlap")])
def test_dispatch(change, code, says):
    refused("moe_dispatch", DISPATCH, DISPATCH_BASE, change, code, says)


@pytest.mark.parametrize("change,code,says", [
    *[({n: N}, ARG, "null pointer") for n in ("dxp", "inv", "dx")],
    (dict(T=-1), ARG, "bad sizes"), (dict(H=0), ARG, "bad sizes"), (dict(k=0), ARG, "bad sizes"),
    (dict(dt=5), ARG, "type 5"), (dict(dx="dxp"), ARG, "dx overlaps dxp"), (dict(ldxp=-1), ARG, "of dxp"),
    (dict(ldx=3), ARG, "row stride 3 of dx "), (dict(T=1 << 30, k=2), SHAPE, "T*k"),
    (dict(H=(1 << 30) + 1, ldx=1 << 31), SHAPE, "2^30")])
def test_dispatch_backward(change, code, says):
    base = dict(buffers("dxp inv dx"), ldxp=8, dt=F16, T=4, H=8, k=2, ldx=8)
    refused("moe_dispatch_backward", "dxp ldxp dt inv T H k dx ldx", base, change, code, says)


@pytest.mark.parametrize("change,code,says", [
    *[({n: N}, ARG, "null pointer") for n in ("yp", "inv", "wts", "out")],
    (dict(T=-2), ARG, "bad sizes"), (dict(H=0), ARG, "bad sizes"), (dict(k=0), ARG, "bad sizes"),
    (dict(ydt=9), ARG, "unknown type 9"), (dict(odt=9), ARG, "unknown type 9"),
    (dict(ydt=BF16, odt=F32), ARG, "results of type"), (dict(ydt=BF16, odt=F16), ARG, "results of type"),
    (dict(out="yp"), ARG, "out overlaps yp"), (dict(ldyp=-1), ARG, "of yp"), (dict(ldo=7), ARG, "row stride 7 of out"),
    (dict(T=1 << 30, k=2), SHAPE, "T*k"), (dict(H=(1 << 30) + 1, ldo=1 << 31), SHAPE, "2^30")])
def test_combine(change, code, says):
    base = dict(buffers("yp inv wts out"), ldyp=8, ydt=F32, T=4, H=8, k=2, ldo=8, odt=BF16)
    refused("moe_combine", "yp ldyp ydt inv wts T H k out ldo odt", base, change, code, says)


@pytest.mark.parametrize("change,code,says", [
    *[({n: N}, ARG, "null pointer") for n in ("dout", "yp", "inv", "wts")],
    (dict(dyp=N, dwts=N), ARG, "both null"), (dict(dyp="yp"), ARG, "dyp overlaps"),
    (dict(dyp="dout"), ARG, "dyp overlaps"), (dict(T=-1), ARG, "bad sizes"), (dict(H=0), ARG, "bad sizes"),
    (dict(k=0), ARG, "bad sizes"),
    (dict(ydt=7), ARG, "unknown type 7"), (dict(ddt=7), ARG, "unknown type 7"),
    (dict(ydt=F16, ddt=BF16), ARG, "results of type"), (dict(lddout=-1), ARG, "of dout"), (dict(ldyp=-1), ARG, "of yp"),
    (dict(lddyp=4), ARG, "row stride 4 of dyp"), (dict(T=1 << 30, k=2), SHAPE, "T*k"),
    (dict(H=(1 << 30) + 1, lddyp=1 << 31), SHAPE, "2^30")])
def test_combine_backward(change, code, says):
    base = dict(buffers("dout yp inv wts dyp dwts"), lddout=8, ddt=BF16, ldyp=8, ydt=BF16, T=4, H=8, k=2, lddyp=8)
    order = "dout lddout ddt yp ldyp ydt inv wts T H k dyp lddyp dwts"
    refused("moe_combine_backward", order, base, change, code, says)


@pytest.mark.parametrize("change,code,says", [
    *[({n: N}, ARG, "null pointer") for n in ("idx", "wts", "dwts", "dl")],
    (dict(T=-1), ARG, "bad sizes"), (dict(k=0), ARG, "bad sizes"), (dict(k=9), ARG, "bad sizes"),
    (dict(E=300, ld=300), SHAPE, "E=300"), (dict(ld=7), ARG, "row stride 7 of dlogits"), (dict(dt=4), ARG, "type 4"),
    (dict(T=1 << 30), SHAPE, "T*k")])
def test_router_backward(change, code, says):
    base = dict(buffers("idx wts dwts dl"), T=4, E=8, k=2, ld=8, dt=F32)
    refused("moe_route_topk_backward", "idx wts dwts T E k dl ld dt", base, change, code, says)


NORM_SIZES = [(dict(T=-1), ARG, "bad sizes"), (dict(H=0), ARG, "bad sizes"), (dict(H=16385), SHAPE, "H=16385"),
              (dict(dt=3), ARG, "type 3"), (dict(eps=0.0), ARG, "eps"), (dict(eps=-1.0), ARG, "eps"),
              (dict(eps=float("nan")), ARG, "eps"), (dict(eps=float("inf")), ARG, "eps")]


@pytest.mark.parametrize("change,code,says", [
    *NORM_SIZES, (dict(h=N), ARG, "null pointer"), (dict(x=N), ARG, "null pointer"), (dict(ldh=-1), ARG, "of h "),
    (dict(ldx=4), ARG, "row stride 4 of x")])
def test_pre(change, code, says):
    base = dict(buffers("h w x"), ldh=8, dt=BF16, eps=1e-5, T=4, H=8, ldx=8)
    refused("moe_norm_pre", PRE, base, change, code, says)


@pytest.mark.parametrize("change,code,says", [
    *NORM_SIZES, *[({n: N}, ARG, "null pointer") for n in ("dx", "h", "dh")], (dict(lddx=-1), ARG, "of dx"),
    (dict(ldh=-1), ARG, "of h "), (dict(ldr=-1), ARG, "of dres"), (dict(lddh=2), ARG, "row stride 2 of dh"),
    (dict(ws=N), ARG, "workspace of 0"), (dict(wb=16), ARG, "workspace of 16"),
    (dict(ws=ctypes.c_void_p((1 << 40) + 1)), ARG, "aligned")])
def test_pre_backward(change, code, says):
    base = dict(buffers("dx h w dres dh dw ws"), lddx=8, ldh=8, dt=BF16, eps=1e-5, T=4, H=8, ldr=8, lddh=8, wb=1 << 30)
    refused("moe_norm_pre_backward", PRE_BACK, base, change, code, says)


@pytest.mark.parametrize("change,code,says", [
    *NORM_SIZES, *[({n: N}, ARG, "null pointer") for n in ("y", "h", "ho", "xn")],
    (dict(flags=4), ARG, "unknown flags 4"), (dict(mode=4), ARG, "gate mode 4"), (dict(mode=-1), ARG, "gate mode -1"),
    (dict(mode=0), ARG, "do not go together"), (dict(gate=N), ARG, "do not go together"), (dict(ldy=-1), ARG, "of y "),
    (dict(ldh=-1), ARG, "of h "), (dict(ldho=7), ARG, "row stride 7 of h_out"), (dict(ldx=7), ARG, "of x_next"),
    (dict(ldg=-1), ARG, "of gate")])
def test_post(change, code, says):
    refused("moe_norm_post", POST, POST_BASE, change, code, says)


@pytest.mark.parametrize("change,code,says", [
    *NORM_SIZES, *[({n: N}, ARG, "null pointer") for n in ("yp", "inv", "wts", "h", "ho", "xn")],
    (dict(k=0), ARG, "k=0"), (dict(T=1 << 30), SHAPE, "T*k"), (dict(ydt=F16), ARG, "results of type"),
    (dict(ydt=7), ARG, "of type 7"), (dict(dt=F32, ydt=BF16), ARG, "results of type"), (dict(ldyp=-1), ARG, "of yp"),
    (dict(ldyo=7), ARG, "row stride 7 of y_out"), (dict(ldho=7), ARG, "of h_out"), (dict(ho="yp"), ARG, "overlap")])
def test_fused(change, code, says):
    refused("moe_combine_norm_post", FUSED, FUSED_BASE, change, code, says)


@pytest.mark.parametrize("change,code,says", [
    *NORM_SIZES, *[({n: N}, ARG, "null pointer") for n in ("dho", "y", "ho", "dx", "dh", "dy")],
    (dict(flags=8), ARG, "unknown flags 8"), (dict(mode=4), ARG, "gate mode 4"),
    (dict(gate=N), ARG, "do not go together"), (dict(flags=2), ARG, "gradient asked"),
    (dict(flags=1), ARG, "gradient asked"),
    (dict(mode=0, gate=N), ARG, "gradient asked"), (dict(lddho=-1), ARG, "of dh_out"), (dict(ldy=-1), ARG, "of y "),
    (dict(lddh=7), ARG, "row stride 7 of dh "), (dict(lddy=7), ARG, "of dy"), (dict(ldho=-1), ARG, "of h_out"),
    (dict(lddx=-1), ARG, "of dx_next"), (dict(ldg=-1), ARG, "of gate"), (dict(lddg=7), ARG, "of dgate"),
    (dict(ws=N), ARG, "workspace of 0"), (dict(wb=64), ARG, "workspace of 64"),
    (dict(ws=ctypes.c_void_p((1 << 40) + 128)), ARG, "aligned")])
def test_post_backward(change, code, says):
    refused("moe_norm_post_backward", BACK, BACK_BASE, change, code, says)


def test_no_tokens_and_no_buffers():
    """An empty batch's tensors have no address: the calls are valid and launch nothing."""
    def ok(fn, order, base, **change):
        args = {**base, "T": 0, **change}
        assert getattr(q.lib, fn)(*(args[n] for n in order.split()), None) == q.MOE_OK, (
            fn, q.lib.moe_last_error_string())
    rows = "yp inv wts out dout dyp dwts idx dl h x y ho xn yo dho dh dy dx dxp dres"
    none = {n: N for n in rows.split()}
    ok("moe_dispatch_backward", "dxp ld dt inv T H k dx ld", none, ld=8, dt=BF16, H=8, k=2)
    ok("moe_combine", "yp ld dt inv wts T H k out ld dt", none, ld=8, dt=BF16, H=8, k=2)
    ok("moe_combine_backward", "dout ld dt yp ld dt inv wts T H k dyp ld dwts", none, ld=8, dt=BF16, H=8, k=2)
    ok("moe_route_topk_backward", "idx wts dwts T E k dl ld dt", none, E=8, k=2, ld=8, dt=F32)
    ok("moe_norm_pre", PRE, {**none, "w": N}, ldh=8, dt=BF16, eps=1e-5, H=8, ldx=8)
    ok("moe_norm_pre_backward", PRE_BACK, {**none, "w": N, "dw": N, "ws": N}, lddx=8, ldh=8, dt=BF16, eps=1e-5,
       H=8, ldr=8, lddh=8, wb=0)
    for mode in (0, 2, 3):                      # a gate per token or per value is empty too
        ok("moe_norm_post", POST, {**POST_BASE, **none, "gate": N}, mode=mode)
        ok("moe_combine_norm_post", FUSED, {**FUSED_BASE, **none, "gate": N}, mode=mode)
        ok("moe_norm_post_backward", BACK, {**BACK_BASE, **none, "gate": N, "dg": N, "dw": N, "dwn": N}, mode=mode)
