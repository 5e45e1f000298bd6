"""Attention over caches of integers where one position draws nearly all of the weight and some of its
codes are 0, so that those elements are made of the other positions' terms: random calls of
test_kv_attention.py, against its reference and tolerances, chosen for such elements."""
import pytest

import test_kv_attention as tk
from test_kv_attention import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", [1275, 1395, 1539, 1565, 1748, 1940, 2747, 2818, 3068, 3163, 3367, 3422, 3650, 3860, 4449, 4475,
                                  5359, 5533, 5673, 6478, 6718, 7248, 7498, 7914, 8004, 8297, 9253, 9667, 9870, 10389, 11131, 11144,
                                  11213, 11437, 12456, 13022, 13500,
                                  # 8 bits
                                  1454, 1906, 3646, 6473, 6684, 6949, 7435, 7890, 8442, 11381, 11918, 12460, 13075])
def test_random_shapes(seed):
    tk.test_random_shapes(seed)
