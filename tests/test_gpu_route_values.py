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
