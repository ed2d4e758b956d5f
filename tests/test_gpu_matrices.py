"""Products, orthogonalisation and the orthogonalised momentum step over lists of
matrices, against plain forms in 64 bits."""
import pytest
import torch

import fsdp_sharded_optimizer_amd as zs
from tests import matrices_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: ref.FP32, BF16: ref.BF16}


def rand(*shape, seed=0, dtype=F32, std=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


def at_offset(t, off):
    """t's values in a view `off` elements into a buffer."""
    buf = torch.full((t.numel() + off + 64,), float("nan"), dtype=t.dtype, device=t.device)
    view = buf[off:off + t.numel()].view(t.shape)
    view.copy_(t)
    return view, buf


def untouched(buf, off, n):
    return bool(torch.isnan(buf[:off]).all()) and bool(torch.isnan(buf[off + n:]).all())


# m, n, k: single elements, vectors, around the tiles' sides (64, 128, 256) and the k tile's (64), empty sides
PRODUCTS = [(1, 1, 1), (1, 5, 7), (3, 1, 64), (64, 64, 64), (65, 63, 65), (128, 129, 63), (127, 200, 128), (257, 255, 129),
            (256, 256, 192), (0, 5, 3), (5, 0, 3), (4, 6, 0), (300, 8, 640)]


@pytest.mark.parametrize("in_dtype", [BF16, F32])
@pytest.mark.parametrize("c_dtype,d_dtype", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16), (None, F32)])
@pytest.mark.parametrize("ta,tb", [(False, False), (True, False), (False, True), (True, True)])
def test_products(in_dtype, c_dtype, d_dtype, ta, tb):
    alpha, beta = 0.75, -1.5
    a, b, c, d, bufs = [], [], [], [], []
    for i, (m, n, k) in enumerate(PRODUCTS):
        off = i % 3
        a.append(at_offset(rand(*((k, m) if ta else (m, k)), seed=i, dtype=in_dtype), off)[0])
        b.append(at_offset(rand(*((n, k) if tb else (k, n)), seed=100 + i, dtype=in_dtype), off)[0])
        c.append(at_offset(rand(m, n, seed=200 + i, dtype=c_dtype or F32), off)[0])
        out, buf = at_offset(rand(m, n, seed=300 + i, dtype=d_dtype), off)
        d.append(out)
        bufs.append((buf, off, m * n))
    lst = zs.ProductMatrices(a, b, d, c if c_dtype else None, transpose_a=ta, transpose_b=tb)
    zs.product_add_matrices(lst, alpha, beta)
    for (m, n, k), x, y, z, out, where in zip(PRODUCTS, a, b, c, d, bufs):
        x, y = x.t().contiguous() if ta else x, y.t().contiguous() if tb else y
        want = alpha * (x.double() @ y.double()) + (beta * z.double() if c_dtype else 0.0)
        bound = ref.product_bound(x, y, k, alpha, beta, z if c_dtype else None, in_dtype == F32)
        bound = bound + HALF[d_dtype] * (want.abs() + bound)
        assert ((out.double() - want).abs() <= bound).all(), (m, n, k)
        assert untouched(*where), (m, n, k)


@pytest.mark.parametrize("m,n,k", [(512, 3584, 256), (1536, 2048, 192), (2048, 4096, 64)])
@pytest.mark.parametrize("tb", [False, True])
def test_products_of_every_tile_size(m, n, k, tb):
    """Enough tiles for the larger ones, operands read where they lie; in place."""
    a, b = rand(m, k, dtype=BF16), rand(*((n, k) if tb else (k, n)), seed=1, dtype=BF16)
    d = rand(m, n, seed=2)
    c = d.clone()
    lst = zs.ProductMatrices([a], [b], [d], [d], transpose_b=tb)
    assert zs.product_add_matrices_workspace_bytes(lst) == 0
    zs.product_add_matrices(lst, 0.5, 0.25)
    y = b.t().contiguous() if tb else b
    want = 0.5 * (a.double() @ y.double()) + 0.25 * c.double()
    bound = ref.product_bound(a, y, k, 0.5, 0.25, c, False)
    assert ((d.double() - want).abs() <= bound + ref.FP32 * want.abs()).all()


@pytest.mark.parametrize("tb", [False, True])
@pytest.mark.parametrize("m,n,k", [(128, 270, 64), (64, 65, 128), (300, 600, 192), (70, 64, 64)])
def test_products_with_one_operand_copied(m, n, k, tb):
    """One operand is read where it lies, the other needs a copy, either way round, in
    one list (the copy's place then starts where the other operand's would)."""
    a = [rand(m, k, dtype=BF16), at_offset(rand(m, k, seed=1, dtype=BF16), 1)[0], rand(m, k, seed=2, dtype=BF16)]
    b = [rand(*((n, k) if tb else (k, n)), seed=3 + i, dtype=BF16) for i in range(3)]
    if tb:
        b[0] = at_offset(b[0], 1)[0]
    d = [torch.empty(m, n, device="cuda") for _ in range(3)]
    lst = zs.ProductMatrices(a, b, d, transpose_b=tb)
    ws = torch.full((zs.product_add_matrices_workspace_bytes(lst),), 0xFF, dtype=torch.uint8, device="cuda")
    zs.product_add_matrices(lst, workspace=ws)
    for x, y, z in zip(a, b, d):
        y = y.t().contiguous() if tb else y
        want = x.double() @ y.double()
        assert ((z.double() - want).abs() <= ref.product_bound(x, y, k, 1.0, 0.0, None, False) + ref.FP32 * want.abs()).all()


GRAMS = [(1, 1), (1, 9), (9, 1), (64, 64), (65, 70), (70, 65), (129, 300), (300, 129), (257, 64), (5, 0), (0, 4), (256, 512)]


@pytest.mark.parametrize("in_dtype", [BF16, F32])
@pytest.mark.parametrize("d_dtype", [F32, BF16])
@pytest.mark.parametrize("short", [True, False])
def test_grams(in_dtype, d_dtype, short):
    alpha, beta = 0.05, 0.95
    a, d, before, bufs = [], [], [], []
    for i, (r, q) in enumerate(GRAMS):
        a.append(at_offset(rand(r, q, seed=i, dtype=in_dtype), i % 3)[0])
        side = min(r, q) if short else max(r, q)
        s = rand(side, side, seed=50 + i, dtype=d_dtype)
        s = (s + s.t()).contiguous()
        out, buf = at_offset(s, i % 5)
        d.append(out)
        before.append(s)
        bufs.append((buf, i % 5, side * side))
    zs.gram_add_matrices(zs.GramMatrices(a, d, d), alpha, beta)
    for (r, q), x, s, out, where in zip(GRAMS, a, before, d, bufs):
        x = x if x.shape[0] == s.shape[0] else x.t().contiguous()
        xt = x.t().contiguous()
        want = alpha * (x.double() @ xt.double()) + beta * s.double()
        bound = ref.product_bound(x, xt, x.shape[1], alpha, beta, s, in_dtype == F32)
        bound = bound + HALF[d_dtype] * (want.abs() + bound)
        assert ((out.double() - want).abs() <= bound).all(), (r, q)
        assert torch.equal(out, out.t()), (r, q)
        assert untouched(*where), (r, q)


def test_grams_of_larger_tiles():
    for side, k in ((1664, 128), (4992, 64)):
        a = rand(side, k, dtype=BF16)
        d = torch.full((side, side), float("nan"), device="cuda")
        zs.gram_add_matrices(zs.GramMatrices([a], [d]), 2.0, 3.0)
        at = a.t().contiguous()
        want = 2.0 * (a.double() @ at.double())
        assert ((d.double() - want).abs() <= ref.product_bound(a, at, k, 2.0, 0.0, None, False) + ref.FP32 * want.abs()).all()
        assert torch.equal(d, d.t())


@pytest.mark.parametrize("dtype,tb", [(BF16, False), (BF16, True), (F32, False), (F32, True)])
def test_products_beyond_32_bits(dtype, tb):
    """The longest k, and operands of more bytes than 32 bits address."""
    m, n, k = 9, 2040, 1 << 20
    a, b = rand(m, k, seed=1, dtype=dtype), rand(*((n, k) if tb else (k, n)), seed=2, dtype=dtype)
    d = torch.empty(m, n, dtype=F32, device="cuda")
    zs.product_add_matrices(zs.ProductMatrices([a], [b], [d], transpose_b=tb))
    want = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for at in range(0, k, k // 16):
        y = b[:, at:at + k // 16].t().contiguous() if tb else b[at:at + k // 16]
        want += a[:, at:at + k // 16].double() @ y.double()
    # An addition is off by 2^-24 of the running sum at most, and that is no larger, rms, than
    # the result: k errors (3 k of split inputs) of either sign add up to sqrt(k) of one.  A
    # split product is off by 3 * 2^-16 of itself at most; their errors add up as the products do.
    split = dtype == F32
    assert ref.far(d, want) <= ((3 if split else 1) * k) ** 0.5 * ref.FP32 + (3 * 2.0 ** -16 if split else 0.0)


def test_products_of_non_finite_inputs():
    """An infinity or NaN stays in its row and column; masked out by beta = 0 in c."""
    a, b = rand(70, 100, dtype=BF16), rand(100, 90, seed=1, dtype=BF16)
    a[3, 5], b[7, 80], a[69, 99] = float("inf"), float("nan"), float("-inf")
    c = torch.full((70, 90), float("nan"), device="cuda")
    d = torch.empty(70, 90, device="cuda")
    zs.product_add_matrices(zs.ProductMatrices([a], [b], [d], [c]), 1.0, 0.0)
    bad = ~torch.isfinite(d)
    want = torch.zeros_like(bad)
    want[3], want[69], want[:, 80] = True, True, True
    assert torch.equal(bad, want)
    fine = torch.isfinite(d)
    full = torch.where(torch.isfinite(a), a, 0).double() @ torch.where(torch.isfinite(b), b, 0).double()
    assert ((d.double() - full).abs()[fine] < 1e-3).all()
    assert torch.isinf(d[3][torch.isfinite(b[5].float()) & (b[5] != 0) & ~bad[0]]).all()


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (63, 65), (64, 64), (128, 64), (100, 257), (251, 683), (683, 251), (256, 600), (320, 320)]


@pytest.mark.parametrize("kind", ["noise", "directions", "rank one", "fading"])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalize(kind, dtype):
    x, y, bufs = [], [], []
    for i, (r, c) in enumerate(SHAPES):
        x.append(at_offset(ref.matrix(r, c, i, kind, dtype), i % 4)[0])
        out, buf = at_offset(torch.zeros(r, c, dtype=BF16, device="cuda"), i % 3)
        y.append(out)
        bufs.append((buf, i % 3, r * c))
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(x, y))
    for s, a, b, where in zip(SHAPES, x, y, bufs):
        assert ref.far(b, ref.orthogonal(a)) <= ref.NS_BOUND + ref.BF16, s
        assert untouched(*where), s


@pytest.mark.parametrize("steps,coefficients", [(1, ref.COEFFICIENTS), (2, ref.COEFFICIENTS), (3, (1.5, -0.5, 0.0)), (8, (1.875, -1.25, 0.375))])
def test_orthogonalize_other_polynomials(steps, coefficients):
    x = [ref.matrix(r, c, 7) for r, c in ((96, 200), (130, 70))]
    y = [torch.empty_like(t, dtype=BF16) for t in x]
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(x, y), steps=steps, coefficients=coefficients)
    for a, b in zip(x, y):
        assert ref.far(b, ref.orthogonal(a, steps, coefficients)) <= ref.NS_BOUND + ref.BF16


@pytest.mark.parametrize("kind", ["noise", "directions", "rank one", "fading"])
@pytest.mark.parametrize("short,long", [(8, 4096), (16, 11008), (33, 1025), (64, 140000), (64, 65)])
def test_orthogonalize_skinny_matrices(kind, short, long):
    """Both ways round, more columns than one partial sum, more than 128 of them."""
    x = [ref.matrix(short, long, 5, kind), ref.matrix(long, short, 6, kind)]
    y = [torch.empty_like(t, dtype=BF16) for t in x]
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(x, y))
    for a, b in zip(x, y):
        assert ref.far(b, ref.orthogonal(a)) <= ref.NS_BOUND + ref.BF16


@pytest.mark.parametrize("short,long", [(1, 1), (1, 9), (2, 3), (16, 40), (64, 300)])
def test_muon_step_of_skinny_matrices_in_full_precision(short, long):
    """p = -step O from p = 0 shows O in fp32: no fp16 rounding is in it."""
    for rows, cols in ((short, long), (long, short)):
        g = ref.matrix(rows, cols, 3)
        p, m = torch.zeros(rows, cols, device="cuda"), torch.zeros(rows, cols, device="cuda")
        zs.muon_step_matrices(zs.MuonConfig(lr=1.0), zs.MuonMatrices([p], [g], [m], scale=1.0))
        assert ref.far(-p, ref.orthogonal(g)) <= 1e-4


def test_orthogonalize_is_near_the_polar_factor():
    x = ref.matrix(384, 512, 1)
    y = torch.empty_like(x, dtype=BF16)
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices([x], [y]), steps=12, coefficients=(1.875, -1.25, 0.375))
    u, s, v = torch.linalg.svd(x.double(), full_matrices=False)
    assert float(s[-1] / s[0]) > 0.02          # the polynomial multiplies small values by 1.875 a step
    assert ref.far(y, u @ v) < 0.02


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_orthogonalize_zero_tiny_huge_and_non_finite(dtype):
    base = ref.matrix(70, 90, 3)
    x = [torch.zeros(70, 90, device="cuda", dtype=dtype), (base * 1e-20).to(dtype), (base * 1e30).to(dtype), base.to(dtype).clone(),
         base.to(dtype).clone(), base.to(dtype)]
    x[3][4, 4], x[4][69, 89] = float("nan"), float("inf")
    y = [torch.empty_like(t, dtype=BF16) for t in x]
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(x, y), eps=1e-25)
    assert not y[0].any() and torch.isnan(y[3]).all() and torch.isnan(y[4]).all()
    for k in (1, 2, 5):
        assert ref.far(y[k], ref.orthogonal(x[k].double(), eps=1e-25)) <= ref.NS_BOUND + ref.BF16, k
    # below eps the matrix stays small: X = in / eps
    small = [(base * 1e-7).to(dtype)]
    out = [torch.empty_like(small[0], dtype=BF16)]
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(small, out), eps=1.0)
    assert ref.far(out[0], ref.orthogonal(small[0].double(), eps=1.0)) <= ref.NS_BOUND + ref.BF16


def muon_case(shapes, param, grad, copy, seed=0):
    p = [(ref.matrix(r, c, seed + i) * 20).to(param) for i, (r, c) in enumerate(shapes)]
    g = [ref.matrix(r, c, seed + 100 + i, "directions", grad) for i, (r, c) in enumerate(shapes)]
    m = [ref.matrix(r, c, seed + 200 + i, "directions") * 0.01 for i, (r, c) in enumerate(shapes)]
    b = [torch.zeros(r, c, dtype=BF16, device="cuda") for r, c in shapes] if copy else None
    return p, g, m, b


@pytest.mark.parametrize("param,grad,copy", [(F32, BF16, True), (F32, F32, False), (BF16, BF16, False), (BF16, F32, False)])
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("clip", [True, False])
def test_muon_step(param, grad, copy, nesterov, clip):
    p, g, m, b = muon_case(SHAPES, param, grad, copy)
    lists = {"p": p, "g": g, "m": m}
    held = {k: [at_offset(t, i % 4) for i, t in enumerate(ts)] for k, ts in lists.items()}
    P, G, M = ([t for t, _ in held[k]] for k in "pgm")
    norm = sum((t.float() * 0.125).double().square().sum() for t in g).reshape(1)
    hp = zs.MuonConfig(lr=0.02, momentum=0.9, nesterov=nesterov, weight_decay=0.1, grad_scale=0.125,
                       max_norm=0.5 * float(norm.sqrt()) if clip else 0.0)
    zs.muon_step_matrices(hp, zs.MuonMatrices(P, G, M, b, scale="spectral"), norm_sq=norm if clip else None)
    coef = float((hp.max_norm / (norm.sqrt() + 1e-6)).clamp(max=1.0).float()) if clip else 1.0
    for i, (r, c) in enumerate(SHAPES):
        new, u = ref.momentum(m[i], g[i], 0.9, nesterov, 0.125, coef)
        assert torch.equal(M[i], new), (r, c)
        o = ref.orthogonal(u)
        step = 0.02 * max(1.0, r / c) ** 0.5
        want = p[i].double() * (1 - 0.02 * 0.1) - step * o
        slack = ref.NS_BOUND * step * float(o.norm()) + 4 * ref.FP32 * float(p[i].double().norm() + step * o.norm())
        assert float((P[i].double() - want).norm()) <= slack + HALF[param] * float(want.norm()), (r, c)
        if copy:
            assert torch.equal(b[i], P[i].to(BF16)), (r, c)
        assert torch.equal(G[i], g[i])
    for ts in held.values():
        for i, (t, buf) in enumerate(ts):
            assert untouched(buf, i % 4, t.numel())


def test_muon_step_on_a_non_finite_norm_changes_nothing():
    for value in (float("nan"), float("inf")):
        p, g, m, b = muon_case(SHAPES[:8], F32, BF16, True)
        before = [t.clone() for t in p + m + b]
        zs.muon_step_matrices(zs.MuonConfig(lr=0.02), zs.MuonMatrices(p, g, m, b),
                              norm_sq=torch.tensor([value], dtype=torch.float64, device="cuda"))
        assert all(torch.equal(x, y) for x, y in zip(before, p + m + b))


def test_muon_step_with_device_scalars_is_the_same():
    p, g, m, b = muon_case(SHAPES, F32, BF16, True)
    q, h, n, c = muon_case(SHAPES, F32, BF16, True)
    hp = zs.MuonConfig(lr=0.02, weight_decay=0.1, grad_scale=0.5, max_norm=1e-3)
    norm = torch.ones(1, dtype=torch.float64, device="cuda")
    zs.muon_step_matrices(hp, zs.MuonMatrices(p, g, m, b), norm_sq=norm)
    sc = torch.frombuffer(bytearray(zs.muon_scalars_bytes(hp)), dtype=torch.uint8).cuda()
    zs.muon_step_matrices_dev(sc, 5, zs.MuonMatrices(q, h, n, c), norm_sq=norm)
    assert all(torch.equal(x, y) for x, y in zip(p + m + b, q + n + c))


def test_long_lists_and_groups_equal_single_calls():
    """More matrices than a table holds, and more elements than share the workspace: each
    matrix gets the bits that it gets alone (products do not depend on a launch's tiles
    beyond their size, which the test holds fixed by comparing lists of one tile size)."""
    shapes = [(40, 30 + i % 7) for i in range(700)]
    p, g, m, _ = muon_case(shapes, F32, BF16, False)
    q, h, n, _ = muon_case(shapes, F32, BF16, False)
    hp = zs.MuonConfig(lr=0.02)
    zs.muon_step_matrices(hp, zs.MuonMatrices(p, g, m))
    zs.muon_step_matrices(hp, zs.MuonMatrices(p, g, m))
    for a in range(0, 700, 50):
        part = zs.MuonMatrices(q[a:a + 50], h[a:a + 50], n[a:a + 50])
        zs.muon_step_matrices(hp, part)
        zs.muon_step_matrices(hp, part)
    for x, y in zip(p + m, q + n):
        assert ref.far(x, y) <= 2 * ref.NS_BOUND     # tiles of another size add in another order
    assert all(torch.equal(x, y) for x, y in zip(m, n))


def test_a_group_larger_than_the_shared_workspace():
    shapes = [(8192, 28672), (64, 64), (28672, 8192), (8192, 28672), (1024, 4096)]
    x = [ref.matrix(r, c, i, "directions", BF16) for i, (r, c) in enumerate(shapes)]
    y = [torch.empty_like(t) for t in x]
    lst = zs.OrthogonalizeMatrices(x, y)
    need = zs.orthogonalize_matrices_workspace_bytes(lst)
    # two of the large ones share it: each X's two halves twice, and two of 8192 x 8192
    assert 2 * 2 * (4 * 8192 * 28672 + 2 * 8192**2) < need < 2.02 * 2 * (4 * 8192 * 28672 + 2 * 8192**2)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")      # NaN patterns
    zs.orthogonalize_matrices(lst, workspace=ws)
    for a, b in zip(x, y):
        assert ref.far(b, ref.orthogonal(a)) <= ref.NS_BOUND + ref.BF16, tuple(a.shape)


@pytest.mark.parametrize("shape", [(2040, 1 << 20), (1 << 20, 2040), (46300, 46300 // 64)])
def test_orthogonalize_beyond_32_bits(shape):
    """The longest sides, and more bytes than 32 bits address."""
    x = rand(*shape, seed=5, dtype=BF16)
    y = torch.empty_like(x)
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices([x], [y]))
    assert ref.far(y, ref.orthogonal(x)) <= ref.NS_BOUND + ref.BF16


@pytest.mark.parametrize("shapes", [[(1024, 1024)], [(1024, 1025)], [(1024, 1024), (300, 40), (1024, 1025), (64, 16384), (16385, 64), (7, 9)],
                                    [(90, 90 + i % 5) for i in range(130)] + [(64, 16384)]])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_norms_of_few_and_of_many_partial_sums(shapes, dtype):
    """Up to 2^20 elements a matrix's norm is formed where it is used, above by a launch
    of its own, for all matrices of the call."""
    x = [ref.matrix(r, c, i, "directions", dtype) * 2.0 ** (i % 5 - 2) for i, (r, c) in enumerate(shapes)]
    y = [torch.empty_like(t, dtype=BF16) for t in x]
    zs.orthogonalize_matrices(zs.OrthogonalizeMatrices(x, y))
    for s, a, b in zip(shapes, x, y):
        assert ref.far(b, ref.orthogonal(a)) <= ref.NS_BOUND + ref.BF16, s


def test_same_call_same_bits():
    out = []
    for _ in range(3):
        p, g, m, b = muon_case(SHAPES, F32, BF16, True)
        zs.muon_step_matrices(zs.MuonConfig(lr=0.02), zs.MuonMatrices(p, g, m, b))
        out.append(p + m + b)
    assert all(torch.equal(x, y) for other in out[1:] for x, y in zip(out[0], other))


def test_stacks_are_lists_of_their_matrices():
    p, g, m, _ = muon_case([(96, 160)] * 4, F32, F32, False)
    stack = [torch.stack(ts) for ts in (p, g, m)]
    zs.muon_step_matrices(zs.MuonConfig(lr=0.02), zs.MuonMatrices(p, g, m))
    zs.muon_step_matrices(zs.MuonConfig(lr=0.02), zs.MuonMatrices(*[[s] for s in stack]))
    assert torch.equal(stack[0], torch.stack(p)) and torch.equal(stack[2], torch.stack(m))


def test_calls_on_another_stream():
    a, d = ref.matrix(300, 200, 1, dtype=BF16), torch.zeros(300, 300, device="cuda")
    p, g, m, b = muon_case(SHAPES, F32, BF16, True)
    q, h, n, c = muon_case(SHAPES, F32, BF16, True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        zs.gram_add_matrices(zs.GramMatrices([a], [d]))
    zs.muon_step_matrices(zs.MuonConfig(lr=0.02), zs.MuonMatrices(p, g, m, b), stream=side)
    side.synchronize()
    e = torch.zeros(300, 300, device="cuda")
    zs.gram_add_matrices(zs.GramMatrices([a], [e]))
    zs.muon_step_matrices(zs.MuonConfig(lr=0.02), zs.MuonMatrices(q, h, n, c))
    assert torch.equal(d, e) and all(torch.equal(x, y) for x, y in zip(p + m + b, q + n + c))
