"""GPU parity of the router's choice (include/ffn_experts.h) at values where an
order of bits, or a sum in fp32, is not that of the numbers, against the fp64
definition (oracle/experts_oracle.py). Choices are compared as whole numbers, the
weights and scores within the bounds of test_gpu_experts.py.
"""
from __future__ import annotations

import numpy as np
import pytest

from tests.test_gpu_experts import check_route, rng, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def asg(lib):
    return lib


# ---------------------------------------------------------------- zeros of both signs
# experts, top_k, groups, groups that stay: every number of lanes and registers a token
ZEROS = [(8, 3, 2, 1), (16, 5, 4, 2), (32, 5, 4, 2), (64, 8, 8, 4), (60, 8, 5, 3), (128, 8, 16, 5), (256, 8, 8, 4), (250, 16, 10, 6)]


def zeros(g, m, experts, rest):
    """Rows whose largest logits are zeros of both signs, in any order."""
    l = -np.abs(g.normal(0, 2, (m, experts))) - 0.5
    if rest == "none":
        l[:] = -np.inf
    zero = np.where(g.random((m, experts)) < 0.5, -0.0, 0.0)
    l = np.where(g.random((m, experts)) < 0.3, zero, l)
    l[0] = zero[0]                                      # a row times a mask of 0: nothing but zeros
    l[1] = np.where(np.arange(experts) % 2, 0.0, -0.0)
    l[2] = np.where(np.arange(experts) == experts - 1, 0.0, -0.0)
    return l


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("m", [33, 1040])
@pytest.mark.parametrize("shape", ZEROS, ids=lambda s: "x".join(map(str, s)))
def test_zeros_of_both_signs_are_equal(asg, shape, m, dtype):
    experts, top_k, groups, top_groups = shape
    say("route zeros", shape, m, dtype)
    for rest in ("negative", "none"):
        l = zeros(rng(15, m, *shape), m, experts, rest)
        for sigmoid in (False, True):
            check_route(asg, l, dtype, top_k, dict(sigmoid=sigmoid), None)
            check_route(asg, l, dtype, top_k, dict(sigmoid=sigmoid), np.zeros(experts, np.float32))
            for best in (1, 2):
                kw = dict(sigmoid=sigmoid, groups=groups, top_groups=top_groups, group_best=best)
                check_route(asg, l, dtype, top_k, kw, None)


# ---------------------------------------------------------------- biases at the ends of fp32
LOW = float(np.finfo(np.float32).min)
# experts, top_k, groups, groups that stay: groups through LDS, of whole lanes of 16 and of 64
ENDS = [(8, 6, 4, 3), (64, 16, 8, 6), (60, 16, 12, 11), (256, 16, 16, 15), (250, 16, 25, 24)]


@pytest.mark.parametrize("m", [5, 1040])
@pytest.mark.parametrize("shape", ENDS, ids=lambda s: "x".join(map(str, s)))
def test_groups_of_the_lowest_biases_are_groups(asg, shape, m):
    # the sum of two such biases lies below every fp32 number, which is not to have no experts
    experts, top_k, groups, top_groups = shape
    say("route lowest biases", shape, m)
    size, g = experts // groups, rng(16, m, *shape)
    l = g.normal(0, 2, (m, experts))
    l[1, :size] = -np.inf                               # a group that has none
    bias = (0.1 * g.normal(0, 1, experts)).astype(np.float32)
    ends = []
    for n, value in ((2, LOW), (groups, LOW), (top_groups, LOW), (2, -LOW), (groups, -LOW)):
        b = bias.copy()
        b[experts - n * size:] = value                  # the last n groups
        ends.append(b)
    b = bias.copy()
    b[-size], b[-2 * size:-size] = LOW, LOW             # one of a group's two, and both of another's
    b[-3 * size:-2 * size] = LOW / 2                    # whose sum is the lowest number itself
    ends.append(b)
    ends.append(-b)
    for b in ends:
        for sigmoid in (False, True):
            for best in (1, 2):
                check_route(asg, l, "f32", top_k, dict(sigmoid=sigmoid, groups=groups, top_groups=top_groups, group_best=best), b)
            check_route(asg, l, "f32", top_k, dict(sigmoid=sigmoid), b)
