"""Every tile size of the calls over matrices, with several k tiles, ragged sides and every
output, against plain forms in 64 bits; lists longer than a launch's table."""
import pytest
import torch

import fsdp_sharded_optimizer_amd as zs
from tests import matrices_reference as ref
from tests import matrices_tiles as tiles

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: ref.FP32, BF16: ref.BF16}


def rand(*shape, seed=0, dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=gen, device="cuda").to(dtype)


@pytest.mark.parametrize("shape,side", tiles.PRODUCTS)
@pytest.mark.parametrize("in_dtype,d_dtype", [(BF16, F32), (BF16, BF16), (F32, F32)])
@pytest.mark.parametrize("tb", [False, True])
def test_products(shape, side, in_dtype, d_dtype, tb):
    """Twice, in place: the residual is the result's own buffer."""
    m, n, k = shape
    a, b = rand(m, k, dtype=in_dtype), rand(*((n, k) if tb else (k, n)), seed=1, dtype=in_dtype)
    d = rand(m, n, seed=2, dtype=d_dtype)
    c = d.clone()
    lst = zs.ProductMatrices([a], [b], [d], [d], transpose_b=tb)
    assert (zs.product_add_matrices_workspace_bytes(lst) == 0) == (in_dtype == BF16)
    zs.product_add_matrices(lst, 0.5, 0.25)
    y = b.t().contiguous() if tb else b
    want = 0.5 * (a.double() @ y.double()) + 0.25 * c.double()
    bound = ref.product_bound(a, y, k, 0.5, 0.25, c, in_dtype == F32)
    assert ((d.double() - want).abs() <= bound + HALF[d_dtype] * (want.abs() + bound)).all()


@pytest.mark.parametrize("shape,side", tiles.GRAMS)
@pytest.mark.parametrize("in_dtype,d_dtype", [(BF16, F32), (BF16, BF16), (F32, F32), (F32, BF16)])
@pytest.mark.parametrize("turned", [False, True])
def test_grams(shape, side, in_dtype, d_dtype, turned):
    m, k = shape
    a = rand(*((k, m) if turned else (m, k)), dtype=in_dtype)
    s = rand(m, m, seed=1, dtype=d_dtype)
    s = (s + s.t()).contiguous()
    d = s.clone()
    zs.gram_add_matrices(zs.GramMatrices([a], [d], [d]), 0.05, 0.95)
    x = a.t().contiguous() if turned else a
    xt = x.t().contiguous()
    want = 0.05 * (x.double() @ xt.double()) + 0.95 * s.double()
    bound = ref.product_bound(x, xt, k, 0.05, 0.95, s, in_dtype == F32)
    assert ((d.double() - want).abs() <= bound + HALF[d_dtype] * (want.abs() + bound)).all()
    assert torch.equal(d, d.t())


@pytest.mark.parametrize("in_dtype", [BF16, F32])
def test_both_grams_of_a_square_matrix(in_dtype):
    """What a two-sided preconditioner of a square projection accumulates."""
    a = [rand(n, n, seed=n, dtype=in_dtype) for n in (1, 63, 64, 200)] + [rand(3, 70, 70, seed=7, dtype=in_dtype)]
    for transposed in (False, True):
        d = [torch.full(t.shape, float("nan"), device="cuda") for t in a]
        zs.gram_add_matrices(zs.GramMatrices(a, d, transposed=transposed), 1.0, 0.0)
        for x, y in zip([q for t in a for q in (t if t.dim() == 3 else [t])], [q for t in d for q in (t if t.dim() == 3 else [t])]):
            x = x.t().contiguous() if transposed else x
            xt = x.t().contiguous()
            want = x.double() @ xt.double()
            bound = ref.product_bound(x, xt, x.shape[1], 1.0, 0.0, None, in_dtype == F32)
            assert ((y.double() - want).abs() <= bound + ref.FP32 * (want.abs() + bound)).all()


@pytest.mark.parametrize("shape,square,wide", tiles.STEPS)
@pytest.mark.parametrize("param,copy", [(F32, True), (BF16, False)])
def test_momentum_steps(shape, square, wide, param, copy):
    rows, cols, count = shape
    p = [(ref.matrix(rows, cols, i) * 20).to(param) for i in range(count)]
    g = [ref.matrix(rows, cols, 1000 + i, "directions" if i % 2 else "noise", BF16) for i in range(count)]
    m = [ref.matrix(rows, cols, 2000 + i) * 0.01 for i in range(count)]
    old, mom = [t.clone() for t in p], [t.clone() for t in m]
    b = [torch.zeros(rows, cols, dtype=BF16, device="cuda") for _ in p] if copy else None
    zs.muon_step_matrices(zs.MuonConfig(lr=0.02, momentum=0.9, weight_decay=0.1), zs.MuonMatrices(p, g, m, b, scale=0.5))
    for i in range(count):
        new, u = ref.momentum(mom[i], g[i], 0.9, True)
        assert torch.equal(m[i], new)
        o = ref.orthogonal(u)
        want = old[i].double() * (1 - 0.02 * 0.1) - 0.01 * o
        slack = ref.NS_BOUND * 0.01 * float(o.norm()) + 4 * ref.FP32 * float(old[i].double().norm() + 0.01 * o.norm())
        assert float((p[i].double() - want).norm()) <= slack + HALF[param] * float(want.norm()), i
        if copy:
            assert torch.equal(b[i], p[i].to(BF16)), i


@pytest.mark.parametrize("shape,square,wide", tiles.STEPS)
def test_orthogonalized_outputs(shape, square, wide):
    rows, cols, count = shape
    x = [ref.matrix(rows, cols, i, "directions" if i % 2 else "noise") for i in range(count)]
    y = [torch.empty_like(t, dtype=BF16) for t in x]
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(x, y))
    for i in range(count):
        assert ref.far(y[i], ref.orthogonal(x[i])) <= ref.NS_BOUND + ref.BF16, i


def stepped(shapes, parts):
    """Two steps from parameters of zero over a list in pieces, and its gradients."""
    g = [ref.matrix(r, c, i, dtype=BF16) for i, (r, c) in enumerate(shapes)]
    p = [torch.zeros(r, c, device="cuda") for r, c in shapes]
    m = [torch.zeros(r, c, device="cuda") for r, c in shapes]
    for _ in range(2):
        for at in parts:
            zs.muon_step_matrices(zs.MuonConfig(lr=1.0), zs.MuonMatrices(p[at], g[at], m[at], scale=1.0))
    return p, g


def slices(count, size):
    return [slice(a, a + size) for a in range(0, count, size)]


@pytest.mark.parametrize("shapes,size", [([(40, 30 + i % 7) for i in range(700)], 50),                     # short sides up to 64
                                         ([(70 + i % 9, 65 + i % 31) for i in range(600)], 200),           # 64-wide tiles in each piece too
                                         ([(70, 65 + i % 31) if i % 3 else (1 + i % 64, 90) for i in range(900)], 300)])
def test_lists_longer_than_a_table(shapes, size):
    """A launch's tables hold 118 to 960 matrices: each matrix has the bits that it gets in a
    shorter list, and those are right."""
    p, g = stepped(shapes, [slice(0, len(shapes))])
    q, _ = stepped(shapes, slices(len(shapes), size))
    assert all(torch.equal(x, y) for x, y in zip(p, q))
    for k in range(0, len(shapes), 7):
        # u is 0.0975 and 0.142625 of the gradient: of one direction, which the polynomial takes alone
        want = 2 * ref.orthogonal(g[k])
        assert ref.far(-p[k], want) <= ref.NS_BOUND + 2 ** -20, shapes[k]


@pytest.mark.parametrize("steps", [8, 12, 32])
def test_many_steps_stay_bounded(steps):
    """Of matrices without full rank, short sides above 64: the polynomial keeps [0, 1.2017] in
    itself, and brings what is up to 0.05 above back (f(1.25) = 1.18); a step is off by less.
    The last one may leave it by what the result is off by."""
    x = [ref.matrix(96, 200, 1, "rank one"), ref.matrix(300, 70, 2, "rank one", BF16).float(), ref.matrix(300, 500, 3, "directions"),
         rand(128, 3, seed=4) @ rand(3, 256, seed=5), torch.ones(65, 65, device="cuda")]
    y = [torch.empty_like(t, dtype=BF16) for t in x]
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(x, y), steps=steps)
    for b in y:
        assert torch.isfinite(b).all()
        b = b.double()
        assert float(torch.linalg.matrix_norm(b, 2)) <= 1.2017 + (ref.NS_BOUND + ref.BF16) * float(b.norm()), tuple(b.shape)
