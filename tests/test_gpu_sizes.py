"""Sizes that int32 does not hold are refused: a call by the C ABI would see them
cut off, and do a part of the work in silence."""
from __future__ import annotations

import pytest

from tests.test_gpu_experts import say, torch_

pytestmark = pytest.mark.gpu
MANY = 2 ** 32 + 8                    # cut off: 8


@pytest.fixture(scope="module")
def asg(lib):
    return lib


def test_numbers_past_int32(asg):
    say("numbers past int32")
    torch = torch_()
    l, ids = torch.zeros(4, 64, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    off = torch.zeros(9, dtype=torch.int32, device="cuda")
    for call in (lambda: asg.route_forward(l, MANY, weights=l, ids=ids), lambda: asg.route_forward(l, 2, groups=MANY),
                 lambda: asg.route_forward(l, 2, groups=8 - 2 ** 32), lambda: asg.route_forward(l, 2, groups=-8),
                 lambda: asg.route_forward(l, 2, groups=8, top_groups=MANY), lambda: asg.route_forward(l, 2, group_best=2 ** 32 + 1),
                 lambda: asg.group_rows(ids, MANY, offsets=off)):
        with pytest.raises(ValueError):
            call()


def test_rows_past_int32(asg):
    # 17 GB of int32 and half as many of logits, hardly any of it written
    say("rows past int32")
    torch = torch_()
    ids = torch.empty(MANY, dtype=torch.int32, device="cuda")
    small = torch.empty(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="sizes are"):
        asg.group_rows(ids, 4, rows=ids, slots=ids)
    logits = torch.empty(MANY, 1, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="sizes are"):
        asg.route_forward(logits, 1, weights=ids.view(torch.float32).view(MANY, 1), ids=ids.view(MANY, 1))
    with pytest.raises(ValueError, match="sizes are"):
        asg.route_backward(logits, ids.view(MANY, 1), ids.view(torch.float32).view(MANY, 1), dlogits=logits)
    assert asg.group_rows(small, 4)[0].shape == (5,)    # what fits is taken
