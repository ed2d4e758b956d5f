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


def growth(x, steps, coefficients):
    """What an error of every step's X, relative in the Frobenius norm, adds up to in the
    result, to first order: in the singular vectors' basis a step multiplies an
    error's symmetric part by (f(s) - f(t)) / (s - t), the other part by (f(s) + f(t)) / (s +
    t), and what lies outside the right ones' span by f(s) / s."""
    a, b, c = coefficients
    s = torch.linalg.svdvals(x.double() / x.double().norm())
    factors, norms = [], [s.norm()]
    for _ in range(steps):
        y = a * s + b * s**3 + c * s**5
        apart = s[:, None] - s[None]
        slope = (a + 3 * b * s**2 + 5 * c * s**4)[:, None].expand(len(s), len(s))
        even = torch.where(apart.abs() > 1e-9, (y[:, None] - y[None]) / torch.where(apart == 0, 1.0, apart), slope)
        factors.append((even.abs(), (y[:, None] + y[None]).abs() / (s[:, None] + s[None]), (y / s).abs()))
        s = y
        norms.append(s.norm())
    total, product = 0.0, [torch.ones_like(f) for f in factors[-1]]
    for k in reversed(range(steps)):
        product = [p * f for p, f in zip(product, factors[k])]
        total += max(float(p.max()) for p in product) * float(norms[k] / norms[-1])
    return total


def low_rank(rows, cols, rank, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    return r(rows, rank) @ r(rank, cols) * 1e-3


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 5, 6, 7, 8, 10, 11, 12])
def test_steps_of_ill_conditioned_matrices_follow_the_formula(steps):
    """Singular values down to 1e-3 of the largest: a step's roundings (2^-20 together) grow as
    growth() says.  S is rounded to 2^-23 of its largest value; in small directions it is off
    by more, NS_BOUND's derivation says by how much in five steps, and that grows no further."""
    x = [low_rank(64, 256, 8, 1).to(BF16).float(), ref.matrix(40, 130, 2, "directions"), ref.matrix(130, 40, 2, "directions"),
         ref.matrix(33, 200, 3, "fading"), ref.matrix(64, 1100, 4, "directions"), ref.matrix(64, 70, 5)]
    for a, b in zip(x, orthogonalized(x, steps)):
        bound = growth(a, steps, ref.COEFFICIENTS) * 2.0 ** -20 + ref.NS_BOUND + ref.BF16
        assert ref.far(b, ref.orthogonal(a, steps)) <= bound, tuple(a.shape)


@pytest.mark.parametrize("steps", [8, 10, 12, 20, 32])
def test_null_directions_stay_bounded(steps):
    """Of a matrix without full rank what the steps make of its null directions is what
    roundings left there, but the polynomial keeps [0, 1.2017] in itself: no singular
    value leaves that by more than the result is off by."""
    x = [ref.matrix(48, 96, 3, "rank one"), low_rank(128, 16, 4, 2), low_rank(64, 300, 1, 3),
         ref.matrix(64, 2000, 4, "rank one").to(BF16).float()]
    for b in orthogonalized(x, steps):
        assert torch.isfinite(b).all()
        b = b.double()
        assert float(torch.linalg.matrix_norm(b, 2)) <= 1.2017 + (ref.NS_BOUND + ref.BF16) * float(b.norm())


@pytest.mark.parametrize("coefficients,steps", [((4.0848, -6.8946, 2.927), 5), ((4.0848, -6.8946, 2.927), 6),
                                                ((5.0, -20.0, 16.0), 5), ((8.0, -20.0, 12.0), 3), ((12.0, -8.0, 1.0), 2), ((32.0, 0.0, 0.0), 1)])
def test_steeper_polynomials(coefficients, steps):
    """Fewer steps at a time, the steeper the polynomial is at 0."""
    x = [ref.matrix(40, 130, 2, "directions"), ref.matrix(300, 64, 3, "fading"), ref.matrix(9, 100, 4), ref.matrix(64, 1100, 5, "directions")]
    for a, b in zip(x, orthogonalized(x, steps, coefficients)):
        bound = growth(a, steps, coefficients) * 2.0 ** -20 + ref.NS_BOUND + ref.BF16
        assert ref.far(b, ref.orthogonal(a, steps, coefficients)) <= bound, tuple(a.shape)


@pytest.mark.parametrize("coefficients,steps", [(ref.COEFFICIENTS, 7), ((4.0848, -6.8946, 2.927), 5)])
def test_long_matrices(coefficients, steps):
    """Several columns to a partial sum, and more than 128 sums' worth of them."""
    x = [ref.matrix(64, 140000, 1), ref.matrix(33000, 20, 2), ref.matrix(7, 2049, 3)]
    for a, b in zip(x, orthogonalized(x, steps, coefficients)):
        bound = growth(a, steps, coefficients) * 2.0 ** -20 + ref.NS_BOUND + ref.BF16
        assert ref.far(b, ref.orthogonal(a, steps, coefficients)) <= bound, tuple(a.shape)


@pytest.mark.parametrize("coefficients,steps,same", [(ref.COEFFICIENTS, 11, True), ((4.0848, -6.8946, 2.927), 6, False),
                                                     ((5.0, -20.0, 16.0), 5, False)])
def test_momentum_steps_with_device_scalars(coefficients, steps, same):
    """The bits of the call with host scalars; for a polynomial that takes fewer steps at a
    time (the launches cannot go by a coefficient in device memory) both by the formula."""
    shapes = [(64, 64), (3, 500), (500, 40), (96, 80), (1, 1), (64, 3000)]
    hp = zs.MuonConfig(lr=0.02, ns_steps=steps, coefficients=coefficients)
    out = []
    for dev in (False, True):
        p = [ref.matrix(r, c, i) for i, (r, c) in enumerate(shapes)]
        g = [ref.matrix(r, c, 10 + i, dtype=BF16) for i, (r, c) in enumerate(shapes)]
        m = [torch.zeros_like(t) for t in p]
        lst = zs.MuonMatrices(p, g, m)
        if dev:
            sc = torch.frombuffer(bytearray(zs.muon_scalars_bytes(hp)), dtype=torch.uint8).cuda()
            zs.muon_step_matrices_dev(sc, steps, lst)
        else:
            zs.muon_step_matrices(hp, lst)
        out.append(p + m)
        for i, (r, c) in enumerate(shapes):
            assert torch.equal(m[i], ref.momentum(torch.zeros(r, c, device="cuda"), g[i], 0.95, True)[0])
            u = ref.momentum(torch.zeros(r, c, device="cuda"), g[i], 0.95, True)[1]
            o, old = ref.orthogonal(u, steps, coefficients), ref.matrix(r, c, i).double()
            want = old - 0.02 * 0.2 * max(r, c) ** 0.5 * o
            off = growth(u, steps, coefficients) * 2.0 ** -20 + ref.NS_BOUND
            step = 0.02 * 0.2 * max(r, c) ** 0.5 * float(o.norm())
            if min(r, c) <= 64:
                assert float((p[i].double() - want).norm()) <= off * step + 4 * ref.FP32 * (float(old.norm()) + step), (r, c)
    assert all(torch.equal(a, b) for a, b in zip(*out)) or not same
