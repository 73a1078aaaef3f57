"""The examples' own checks fail on what they are there to find: a NaN among the results, a stage that is off (no GPU
needed)."""
import importlib.util
import math
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load(name):
    spec = importlib.util.spec_from_file_location("example_" + name, os.path.join(ROOT, "examples", name + ".py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def spoilt(t, value):
    t = t.clone()
    t.view(-1)[3] = value
    return t


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("first", [False, True])
def test_decoder_layer_check_fails_on_a_stage_that_is_not_finite(value, first):
    E = load("decoder_layer")
    want = torch.randn((4, 16), dtype=torch.float64)
    right = want.bfloat16()
    fine, bad = {"norm": E.rel(right, want)}, {"norm": E.rel(spoilt(right, value), want)}
    worst = {}
    for found in (bad, fine) if first else (fine, bad):
        E.gather(worst, found)
    assert E.off_limits(worst) == ["norm"]
    # the 4-bit norm, which is held to the quantizer's own distance, and a base that is lost as well
    for base in (right, spoilt(right, value)):
        worst = {}
        E.gather(worst, {"norm to 4 bits": E.further(spoilt(right, value), base, want)})
        assert E.off_limits(worst) == ["norm to 4 bits"]
    # a reference that came out NaN says nothing for the result
    assert E.rel(right, spoilt(want, float("nan"))) == math.inf


def test_decoder_layer_check_passes_what_is_right_and_names_what_is_off():
    E = load("decoder_layer")
    want = torch.randn((4, 16), dtype=torch.float64)
    worst = {}
    E.gather(worst, {"rope": E.rel(want.bfloat16(), want), "norm to 4 bits": E.further(want.bfloat16(), want.bfloat16(), want), "sort": 0.0})
    assert E.off_limits(worst) == []
    E.gather(worst, {"rope": E.rel(want * 1.01, want), "sort": float("inf")})
    E.gather(worst, {"rope": 0.0, "sort": 0.0})
    assert sorted(E.off_limits(worst)) == ["rope", "sort"]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_kv_decode_check_fails_on_a_step_that_is_not_finite(value):
    E = load("kv_decode")
    want = torch.randn((4, 16), dtype=torch.float64)
    assert E.rel(spoilt(want.bfloat16(), value), want) == E.rel(want.bfloat16(), spoilt(want, float("nan"))) == math.inf
    assert max(0.0, E.rel(spoilt(want.bfloat16(), value), want)) == math.inf and E.rel(want.bfloat16(), want) <= 2.0 ** -8
