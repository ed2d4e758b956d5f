"""MuonOptimizer: a model's matrices stepped on the library's calls, alone, beside
TensorOptimizer on one norm, resumed and captured."""
import pytest
import torch

import fsdp_sharded_optimizer_amd as zs
from tests import matrices_reference as ref

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
SHAPES = [(64, 192), (300, 100), (3, 96, 130), (8, 200), (128, 128)]


def model(seed=0, dtype=F32):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(*s, generator=gen, device="cuda") * 0.02).to(dtype) for s in SHAPES]


def gradients(step, dtype=BF16):
    gen = torch.Generator(device="cuda").manual_seed(1000 + step)
    return [(torch.randn(*s, generator=gen, device="cuda") * 1e-2).to(dtype) for s in SHAPES]


def plain_step(params, momenta, grads, lr, mu, decays, scale, max_norm):
    """The step in 64 bits; max_norm 0: no clipping."""
    g = [x.double() * scale for x in grads]
    if max_norm:
        norm = sum(x.square().sum() for x in g).sqrt()
        g = [x * min(1.0, float(max_norm / (norm + 1e-6))) for x in g]
    for p, m, x, decay in zip(params, momenta, g, decays):
        m.mul_(mu).add_((1 - mu) * x)
        u = mu * m + (1 - mu) * x
        for q, v in ([(p, u)] if p.dim() == 2 else zip(p, u)):
            q.mul_(1 - lr * decay).sub_(lr * 0.2 * max(v.shape) ** 0.5 * ref.orthogonal(v))


@pytest.mark.parametrize("dtype,grad", [(F32, BF16), (F32, F32), (BF16, BF16)])
@pytest.mark.parametrize("max_norm", [0.0, 0.3])
def test_steps_follow_the_formula(dtype, grad, max_norm):
    p, decays, lr = model(dtype=dtype), [0.1, 0.0, 0.1, 0.0, 0.1], 0.01
    want, mom = [x.double() for x in p], [torch.zeros_like(x, dtype=torch.float64) for x in p]
    copies = [torch.zeros_like(x, dtype=BF16) if k != 1 else None for k, x in enumerate(p)] if dtype == F32 else None
    opt = zs.MuonOptimizer(p, lr=lr, weight_decay=decays, grad_scale=0.5, max_norm=max_norm, param_bf16=copies)
    steps = 4
    for t in range(steps):
        g = gradients(t, grad)
        opt.step(g)
        plain_step(want, mom, g, lr, 0.95, decays, 0.5, max_norm)
    assert opt.t == steps
    for k, (x, y) in enumerate(zip(p, want)):
        update = lr * 0.2 * max(SHAPES[k][-2:]) ** 0.5 * (min(SHAPES[k][-2:]) * (SHAPES[k][0] if len(SHAPES[k]) == 3 else 1)) ** 0.5
        # a step's update is off by NS_BOUND (singular values are at most 1.2); a bf16 parameter rounds every step
        slack = steps * (1.2 * ref.NS_BOUND * update + (ref.BF16 if dtype == BF16 else 4 * ref.FP32) * float(y.norm()))
        assert float((x.double() - y).norm()) <= slack, SHAPES[k]
        if copies and copies[k] is not None:
            assert torch.equal(copies[k], x.to(BF16))
    for x, y in zip(opt.state_dict()["momentum"], mom):
        assert ref.far(x, y) <= 1e-6


def run(opt, params, steps, first=0):
    for t in range(first, first + steps):
        opt.step(gradients(t))
    return [p.clone() for p in params] + [m.clone() for m in opt.state_dict()["momentum"]]


def test_resume_is_bit_exact():
    p, q = model(), model()
    whole = run(zs.MuonOptimizer(p, lr=0.01, max_norm=0.2), p, 5)
    a = zs.MuonOptimizer(q, lr=0.01, max_norm=0.2)
    run(a, q, 2)
    state = {k: [x.cpu() for x in v] if isinstance(v, list) else v for k, v in a.state_dict().items()}
    b = zs.MuonOptimizer(q, lr=0.01, max_norm=0.2)
    b.load_state_dict(state)
    assert b.t == 2 and all(torch.equal(x, y) for x, y in zip(run(b, q, 3, first=2), whole))
    with pytest.raises(ValueError):
        b.load_state_dict({"step": 1, "momentum": state["momentum"][:-1]})
    with pytest.raises(ValueError):
        b.load_state_dict({"step": -1, "momentum": state["momentum"]})


def test_captured_steps_are_the_eager_ones():
    p, q = model(), model()
    eager = zs.MuonOptimizer(p, lr=0.01, weight_decay=[0.1, 0.0, 0.1, 0.0, 0.1], max_norm=0.2)
    other = zs.MuonOptimizer(q, lr=0.01, weight_decay=[0.1, 0.0, 0.1, 0.0, 0.1], max_norm=0.2)
    g = [x.clone() for x in gradients(0)]
    other.bind_grads(g)
    before = [x.clone() for x in q]
    cap = other.capture()
    assert all(torch.equal(x, y) for x, y in zip(q, before)) and other.t == 0
    for t in range(5):
        lr = 0.01 / (t + 1)
        eager.lr = other.lr = lr
        new = gradients(t)
        for x, y in zip(g, new):
            x.copy_(y)
        cap.replay()
        eager.step(new)
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(p + eager._momentum, q + other._momentum)), t
    other.ns_steps = 3
    with pytest.raises(RuntimeError):
        cap.replay()


def test_two_captured_optimizers_replay_in_turn():
    """Each graph has a workspace of its own: replays on two streams at once."""
    ps, opts, caps, want = [], [], [], []
    for k in range(2):
        p = model(k)
        opt = zs.MuonOptimizer(p, lr=0.01)
        opt.bind_grads(gradients(50 + k))
        ps.append(p), opts.append(opt), caps.append(opt.capture())
        q = model(k)
        alone = zs.MuonOptimizer(q, lr=0.01)
        for _ in range(4):
            alone.step(gradients(50 + k))
        want.append(q)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(4):
        for s, cap in zip(streams, caps):
            with torch.cuda.stream(s):
                cap.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for p, q in zip(ps, want) for x, y in zip(p, q))


def test_a_model_on_two_optimizers_and_one_norm():
    """Matrices in bf16 gradients, vectors in fp32 ones: one norm of all clips both steps,
    eagerly and captured; clipping the gradients beforehand gives the same."""
    def build():
        gen = torch.Generator(device="cuda").manual_seed(9)
        vectors = [torch.randn(n, generator=gen, device="cuda") for n in (192, 50, 1)]
        return model(), vectors

    mats, vectors = build()
    mats2, vectors2 = build()
    mats3, vectors3 = build()
    g = gradients(3)
    gv = [torch.randn_like(v) * 1e-2 for v in vectors]
    scale, limit = 0.5, 0.1
    muon = zs.MuonOptimizer(mats, lr=0.01, grad_scale=scale, max_norm=limit)
    adam = zs.TensorOptimizer(vectors, lr=0.01, grad_scale=scale, max_norm=limit)
    norm = torch.zeros(1, dtype=torch.float64, device="cuda")
    norms = torch.zeros(len(g) + len(gv), dtype=torch.float64, device="cuda")
    lst = zs.MixedTensors(g + gv)
    zs.grad_norms_sq_tensors(lst, scale, norm, norms=norms)
    muon.step(g, norm_sq=norm)
    adam.step(gv, norm_sq=norm)
    want = sum((x.double() * scale).square().sum() for x in g + gv)
    assert abs(float(norm) / float(want) - 1) < 1e-12 and float(norm.sqrt()) > limit
    assert torch.allclose(norms.sum(), norm[0], rtol=1e-13)

    # the same with the clipped gradients as tensors
    clipped = [torch.empty_like(x, dtype=F32) for x in g + gv]
    zs.grad_clip_tensors(lst, clipped, scale, limit, norm)
    muon2, adam2 = zs.MuonOptimizer(mats2, lr=0.01), zs.TensorOptimizer(vectors2, lr=0.01)
    muon2.step(clipped[:len(g)])
    adam2.step(clipped[len(g):])
    assert all(torch.equal(x, y) for x, y in zip(mats + vectors, mats2 + vectors2))

    # captured, the norm formed by the caller before each replay
    muon3 = zs.MuonOptimizer(mats3, lr=0.01, grad_scale=scale, max_norm=limit)
    adam3 = zs.TensorOptimizer(vectors3, lr=0.01, grad_scale=scale, max_norm=limit)
    muon3.bind_grads(g)
    adam3.bind_grads(gv)
    caps = muon3.capture(norm_sq=norm), adam3.capture(norm_sq=norm)
    zs.grad_norms_sq_tensors(lst, scale, norm)
    for cap in caps:
        cap.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(mats + vectors, mats3 + vectors3))


def test_a_non_finite_norm_changes_nothing():
    p = model()
    before = [x.clone() for x in p]
    opt = zs.MuonOptimizer(p, lr=0.01, compute_norm=True)
    g = gradients(0)
    g[2][1, 5, 5] = float("nan")
    opt.step(g)
    assert all(torch.equal(x, y) for x, y in zip(p, before)) and not any(m.any() for m in opt._momentum)


def test_refusals():
    p = model()
    for kw in (dict(lr=-1.0), dict(lr=0.1, momentum=1.0), dict(lr=0.1, ns_steps=0), dict(lr=0.1, eps=0.0),
               dict(lr=0.1, coefficients=(40.0, 1.0, 1.0)), dict(lr=0.1, grad_scale=0.0)):
        with pytest.raises(zs.ZShardError):
            zs.MuonOptimizer(p, **kw)
    for kw in (dict(weight_decay=[0.1]), dict(weight_decay=-0.1), dict(max_norm=1.0, compute_norm=False), dict(scale="other"),
               dict(scale=[1.0]), dict(param_bf16=[None])):
        with pytest.raises(ValueError):
            zs.MuonOptimizer(p, lr=0.1, **kw)
    with pytest.raises(ValueError):
        zs.MuonOptimizer([], lr=0.1)
    with pytest.raises(ValueError):
        zs.MuonOptimizer([torch.zeros(5, device="cuda")], lr=0.1)            # a vector
    with pytest.raises(ValueError):
        zs.MuonOptimizer([p[0], p[0][:2]], lr=0.1)                            # the same memory twice
    opt = zs.MuonOptimizer(p, lr=0.1)
    with pytest.raises(RuntimeError):
        opt.step()
    with pytest.raises(RuntimeError):
        opt.capture()
    with pytest.raises(ValueError):
        opt.step([g.t() if g.dim() == 2 else g for g in gradients(0)])        # other shapes
    with pytest.raises(ValueError):
        opt.step([p[0]] + gradients(0, F32)[1:])                              # a gradient in a parameter's memory
    with pytest.raises(TypeError):
        opt.step(gradients(0)[:-1] + gradients(0, F32)[-1:])                  # two dtypes
    with pytest.raises(TypeError):
        opt.step(gradients(0), norm_sq=torch.zeros(1, device="cuda"))


def test_a_refused_step_changes_nothing():
    """What the calls refuse for one weight decay's matrices is refused before another's are
    stepped: a learning rate set later, whose product with the decay does not fit
    binary32, and a factor of it that does not."""
    p = model()
    opt = zs.MuonOptimizer(p, lr=1e-9, weight_decay=[0.0, 1e9, 0.0, 1e9, 0.0])
    opt.lr = 1e30
    before = [x.clone() for x in p + opt._momentum]
    with pytest.raises(zs.ZShardError):
        opt.step(gradients(0))
    assert opt.t == 0 and all(torch.equal(x, y) for x, y in zip(before, p + opt._momentum))
    for scale in (float("inf"), float("nan"), 1e39):
        with pytest.raises(ValueError):
            zs.MuonOptimizer(p, lr=0.01, weight_decay=[0.0, 0.1, 0.0, 0.1, 0.0], scale=[1.0, scale, 1.0, 1.0, 1.0])
        with pytest.raises(ValueError):
            zs.MuonMatrices(p, p, [torch.zeros_like(x) for x in p], scale=scale)
