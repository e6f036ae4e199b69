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
