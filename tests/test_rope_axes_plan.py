"""The axes of a RopeAxes plan, given in any form: the numbers count, not the bytes they are held in."""
import numpy as np
import pytest
import torch

import int8_kv_cache_quant_gb300 as k


@pytest.mark.parametrize("form", [list, tuple, bytes, np.array, lambda a: np.array(a, np.uint8), torch.tensor, iter])
@pytest.mark.parametrize("axes", [[0, 1, 2, 1], [3], [1]])
def test_forms(form, axes):
    plan = k.RopeAxes(torch.zeros(len(axes), dtype=torch.int64), form(axes), 0.5)
    assert list(plan.axis_of) == axes and plan.n_axes == max(axes) + 1 and plan.rotary_dim == 2 * len(axes) and plan.attn_factor == 0.5


@pytest.mark.parametrize("axes", [4, torch.tensor(4), [0, 1, 2, 256], [0, 1, -1, 2], [0, 1, 0.5, 2], "0121"])
def test_what_is_no_list_of_axes_is_refused(axes):
    with pytest.raises((TypeError, ValueError)):
        k.RopeAxes(torch.zeros(4, dtype=torch.int64), axes)
