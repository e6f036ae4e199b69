"""The timed cases of perf/operators.py: drawn ones of every operator and gate go through the package's calls
and give results of the plain forms' shapes and types, whole numbers equal."""
import importlib.util
import os
import random

import pytest
import torch

pytestmark = pytest.mark.gpu

pytest.importorskip("quantized_mixture_experts_grouped_b200")


@pytest.fixture(scope="module")
def ops():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("_timed_cases", os.path.join(root, "perf", "operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def outputs(ops, case, own):
    ops.own = own
    try:
        state = ops.prepare(case, 5)
        return {n: None if v is None else v.clone() for n, v in ops.run(state).items()}
    finally:
        ops.own = False


def kinds(ops):
    """Drawn cases until every operator and every gate of the norms after a block has come up."""
    rng, seen, cases = random.Random(3), set(), []
    while len(seen) < 4 + 3 * 4:
        c = dict(ops.draw(rng), name="")
        kind = c["op"], c.get("gate")
        if kind not in seen:
            seen.add(kind)
            cases.append(c)
    return cases


def test_drawn_cases_of_every_kind(ops):
    for case in kinds(ops):
        want, got = outputs(ops, case, False), outputs(ops, case, True)
        assert want.keys() == got.keys(), case
        for n, w in want.items():
            g = got[n]
            if w is None:
                assert g is None, (case, n)
                continue
            assert g.shape == w.shape and g.dtype == w.dtype, (case, n, g.shape, w.shape)
            if w.is_floating_point():
                assert torch.isfinite(g).all(), (case, n)
            else:
                assert torch.equal(g, w), (case, n)
