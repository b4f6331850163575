"""Tree decode with numbers that are none or without end, against the recurrence along each
path.  Tolerances (relative L2) as in test_gpu_tree.py, with operands rounded to TF32 by 2^-10.5.
"""
import numpy as np
import pytest
import torch

import spec_ref as ref
from test_gpu_tree_range import ROWS, SHAPES, run

pytestmark = pytest.mark.gpu

TOL = {torch.float32: 64 * 2.0 ** -24, torch.bfloat16: 2.0 ** -8 + 8 * 2.0 ** -10.5}
TREE = [-1, 0, 0, 1, 2, 2, 4, -1, 7, 3, 5]          # places 2, 4, 5, 6 and 10 are one branch


@pytest.mark.parametrize("dtype,dims", SHAPES)
@pytest.mark.parametrize("T", [11, 27, 59])
def test_a_reset_by_an_infinite_gate(dtype, dims, T):
    """g = -inf in some channels of a place: alpha = 0 there, and nothing else."""
    d = ref.make_tokens(2, T, 2, *dims, dtype, seed=94)
    parents = torch.tensor([TREE + list(range(10, T - 1))] * 2, dtype=torch.int32)
    d["g"][0, 2, 0, 3] = float("-inf")
    d["g"][1, 4, 1] = float("-inf")
    d["g"][1, 9, 0, ::2] = float("-inf")
    want, _, _ = ref.tree(d, parents)
    assert np.isfinite(want).all()
    out = ref.f64(run(d, parents))
    for n in range(2):
        assert np.linalg.norm(out[n] - want[n]) <= TOL[dtype] * np.linalg.norm(want[n])


@pytest.mark.parametrize("dtype,dims", SHAPES)
@pytest.mark.parametrize("T", [11, 27, 59])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("where", ROWS)
def test_no_number_stays_none_on_its_path(dtype, dims, T, where, bad):
    """NaN or infinity in one row of one place: outputs that are no numbers by the recurrence
    are none here, and other sequences and heads are as the recurrence has them."""
    d = ref.make_tokens(2, T, 2, *dims, dtype, seed=95)
    parents = torch.tensor([TREE + list(range(10, T - 1))] * 2, dtype=torch.int32)
    for n, t, h in ((0, 2, 1), (1, 5, 0)):
        d[where][(n, t, h) + ((9,) if where != "beta" else ())] = bad
    with np.errstate(all="ignore"):
        want, _, _ = ref.tree(d, parents)
    out = ref.f64(run(d, parents))
    fine = np.isfinite(want)
    assert not fine.all() and not np.isfinite(out[~fine]).any()
    for n, h in ((0, 0), (1, 1)):
        a, b = out[n, :, h], want[n, :, h]
        assert np.linalg.norm(a - b) <= TOL[dtype] * np.linalg.norm(b)
