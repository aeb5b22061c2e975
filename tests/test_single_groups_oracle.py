"""Groups of one expert in the float64 definition (CPU)."""
import numpy as np

import oracle


def test_rank_of_a_group_of_one():
    z = np.array([[40.0, 41.0, 0.0]])  # both sigmoids are 1 in 64 bits
    assert oracle.group_gate(z, None, 1, "sigmoid", 3, 1, 1, False, 1.0)[0].tolist() == [[1]]  # ranked by logits
    assert oracle.group_gate(z, None, 1, "sigmoid", 3, 1, 2, False, 1.0)[0].tolist() == [[0]]  # ranked by scores
    assert oracle.group_gate(z, np.zeros(3), 1, "sigmoid", 3, 1, 1, False, 1.0)[0].tolist() == [[0]]
