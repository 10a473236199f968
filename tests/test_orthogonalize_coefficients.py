"""The coefficients of orthogonalize are read in every call (CPU only)."""
import numpy as np
import pytest
import torch

import routing_capacity_dispatch_amd as rcd


@pytest.mark.parametrize("number", [torch.tensor, np.array])
def test_changed_in_place_between_calls(number):
    t = (number(3.0), number(-4.5), number(2.0))
    assert list(rcd._coefficients(t, 2)) == [3.0, -4.5, 2.0] * 2
    t[0][...] = 1.5
    assert list(rcd._coefficients(t, 2)) == [1.5, -4.5, 2.0] * 2
    rows = [list(t), [number(1.0), number(0.5), number(0.25)]]
    assert list(rcd._coefficients(rows, 2)) == [1.5, -4.5, 2.0, 1.0, 0.5, 0.25]
    rows[1][2][...] = 8.0
    assert list(rcd._coefficients(rows, 2)) == [1.5, -4.5, 2.0, 1.0, 0.5, 8.0]
    assert list(rcd._coefficients(number([1.0, 2.0, 4.0]), 1)) == [1.0, 2.0, 4.0]


def test_values_decide_what_is_shared():
    a = rcd._coefficients((1.0, 2.0, 4.0), 3)
    assert rcd._coefficients([torch.tensor(1.0), 2, np.float32(4.0)], 3) is a
    assert rcd._coefficients((1.0, 2.0, 4.5), 3) is not a


@pytest.mark.parametrize("bad", [None, 3.0, "abc", (1.0, 2.0, "x"), (1.0, 2.0, None), ((1.0, 2.0, (3.0,)),),
                                 torch.zeros(2, 3), (torch.zeros(2), 1.0, 2.0), ((1.0, 2.0),) * 2])
def test_what_is_no_number_is_refused(bad):
    with pytest.raises(ValueError, match="coeffs"):
        rcd._coefficients(bad, 2)
