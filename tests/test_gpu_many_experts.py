"""Layers of more than 128 experts on every path, against the oracle: expert ids take all eight bits of a
tile's record."""
import numpy as np
import pytest
import torch

import moe_inputs as mi
from gpu_util import Layer, assert_ffn_close, bf16_dev_to_f32
from test_gpu_bf16 import Bf16Layer, _layer_call
from test_gpu_parity import _run_ffn

pytestmark = pytest.mark.gpu

q = pytest.importorskip("quantized_mixture_experts_grouped_b200")


def every_expert(T, E, k):
    """Logits under which each of T tokens takes the next k experts, so that every expert has some."""
    g = np.random.default_rng(E + T)
    logits = g.standard_normal((T, E)).astype(np.float32)
    for t in range(T):
        logits[t, (t * k + np.arange(k)) % E] += 20.0
    return mi.to_bf16_bits(logits)


@pytest.mark.parametrize("path,T", [("simple", 64), ("grouped", 64), ("grouped", 300), ("sequential", 64), ("decode", 1),
                                    ("decode", 16), ("auto", 64)])
@pytest.mark.parametrize("E", [129, 256])
def test_every_expert_used(path, T, E):
    wl = mi.Workload("many", H=256, I=128, E=E, k=4, T=T)
    layer = Layer(wl, logits=every_expert(T, E, wl.k))
    out, _ = _run_ffn(layer, path)
    assert_ffn_close(bf16_dev_to_f32(out), layer.oracle_out(), f"E={E} T={T} {path}")


def test_permuted_slots_of_many_experts():
    wl = mi.Workload("many", H=256, I=128, E=256, k=4, T=64)
    layer = Layer(wl, logits=every_expert(wl.T, wl.E, wl.k))
    slot = torch.randperm(wl.E, generator=torch.Generator().manual_seed(1))
    d = layer.to_device()
    for n in ("w13", "s13", "w2", "s2"):
        moved = torch.empty_like(d[n])
        moved[slot.cuda()] = d[n]
        d[n] = moved
    out, _ = _run_ffn(layer, "grouped", slot=slot.int().cuda())
    assert_ffn_close(bf16_dev_to_f32(out), layer.oracle_out(), "permuted slots, E=256")


def test_bf16_layer_of_many_experts():
    wl = mi.Workload("many", H=256, I=128, E=256, k=4, T=64)
    layer = Bf16Layer(wl, logits=every_expert(wl.T, wl.E, wl.k))
    got = _layer_call(layer, layer.dev(), q.alloc_workspace(wl.T, wl.H, wl.I, wl.E, wl.k))
    assert_ffn_close(got, layer.oracle_out(), "bf16 E=256")
