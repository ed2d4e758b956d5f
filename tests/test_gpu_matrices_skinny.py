"""Orthogonalisation of matrices whose short side is at most 64, over the polynomials and
numbers of steps that the calls accept, against the formula in 64 bits."""
import pytest
import torch

import fsdp_sharded_optimizer_amd as zs
from tests import matrices_reference as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def orthogonalized(x, steps, coefficients=ref.COEFFICIENTS):
    y = [torch.empty_like(t, dtype=BF16) for t in x]
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(x, y), steps=steps, coefficients=coefficients)
    return y


@pytest.mark.parametrize("coefficients", [(1e-7, 0.0, 0.0), (-2e-7, 1e-8, 0.0), (1e-6, 0.0, 1e-7)])
@pytest.mark.parametrize("steps", [1, 4, 5])
def test_a_polynomial_that_nearly_vanishes(coefficients, steps):
    """The product of the steps' polynomials is down to 1e-35 here: a scale that lifts it
    to 2^13 does not fit binary32.  (The results are about 1e-37 then; those below 2^-126 are off
    by 2^-134 at most, 5e-4 of that.)"""
    x = [ref.matrix(r, c, 7) for r, c in ((64, 200), (90, 8), (1, 30), (64, 64))]
    for a, b in zip(x, orthogonalized(x, steps, coefficients)):
        assert ref.far(b, ref.orthogonal(a, steps, coefficients)) <= ref.NS_BOUND + ref.BF16, tuple(a.shape)


@pytest.mark.parametrize("steps,coefficients", [(16, ref.COEFFICIENTS), (20, ref.COEFFICIENTS), (32, ref.COEFFICIENTS),
                                                (20, (1.5, -0.5, 0.0)), (32, (1.875, -1.25, 0.375))])
def test_many_steps_of_fewer_rows_than_a_tile(steps, coefficients):
    """Well-conditioned matrices: a step multiplies what the steps before it were off by by 0.7
    to 3.4 and, over all of them, the errors of single steps add up to less than 1000 of one
    (first order, from the singular values); a step's few roundings are 2^-22 each: 1e-3."""
    x = [ref.matrix(r, c, 3) for r, c in ((1, 100), (100, 1), (8, 100), (100, 8), (63, 500), (500, 63))]
    for a, b in zip(x, orthogonalized(x, steps, coefficients)):
        assert ref.far(b, ref.orthogonal(a, steps, coefficients)) <= ref.NS_BOUND + ref.BF16, tuple(a.shape)
