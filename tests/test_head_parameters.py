"""Which parameters a model's head is built on, on the CPU: what its calls would
refuse is refused where it is built."""
import types

import pytest
import torch

from optimizer_state_gb300 import build as z3build
from optimizer_state_gb300 import inputs as I
from optimizer_state_gb300 import schedule, z3


def model(*shapes):
    z3build.build()
    w = I.Workload("embed", shapes, 4, 0.02, 1e-3)
    unit = types.SimpleNamespace(w=w, L=z3.Layout(w.numel, w.n_ranks))
    return types.SimpleNamespace(units=[unit], dev=torch.device("cpu"))


@pytest.mark.parametrize("lead,first", [(((13,),), 13), (((2, 2),), 4), (((24,), (3, 5)), 39),
                                        (((1001, 12),), 12012)])
def test_a_parameter_between_boundaries(lead, first):
    """Its weight and gradients would not start on 16 bytes."""
    with pytest.raises(ValueError, match=rf"parameter {len(lead)} of unit 0 starts at element "
                                         rf"{first}: .*multiple of 8"):
        schedule.Head(model(*lead, (1003, 64)), 70, param=len(lead))


@pytest.mark.parametrize("dim", [4, 60, 1001])
def test_rows_between_boundaries(dim):
    with pytest.raises(ValueError, match=rf"parameter 0 of unit 0 has rows of {dim} .*multiple of 8"):
        schedule.Head(model((1003, dim)), 70)
