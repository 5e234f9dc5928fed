"""Argument marshalling of the Python binding, without a GPU."""
import array

import numpy as np
import pytest
import torch

from quantized_kv_cache_15_b200 import kvq


@pytest.mark.parametrize("make", [kvq._ints, kvq._int64s])
@pytest.mark.parametrize("values", [[3, 1, 2], (3, 1, 2), range(3, 0, -1), [3.0, 1.0, 2.7], np.array([3, 1, 2]),
                                    np.array([3.0, 1.0, 2.0]), torch.tensor([3, 1, 2]), torch.tensor([3.0, 1.0, 2.0]),
                                    [np.int64(3), torch.tensor(1), 2.0], [True, False], array.array("q", [3, 1, 2]), []],
                         ids=lambda v: type(v).__name__)
def test_sequences_of_whole_numbers(make, values):
    """Whatever int() takes, element by element."""
    got = make(values)
    assert list(got) == [int(x) for x in values]


def test_numbers_that_do_not_fit_are_refused():
    for make, v in ((kvq._ints, 1 << 31), (kvq._ints, -(1 << 31) - 1), (kvq._int64s, 1 << 63)):
        with pytest.raises(OverflowError):
            make([v])
    with pytest.raises((TypeError, ValueError)):
        kvq._ints(["x"])
    with pytest.raises((TypeError, ValueError)):
        kvq._ints([None])
