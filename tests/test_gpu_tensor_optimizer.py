"""TensorOptimizer (the call-ordering layer over a list) on the GPU: a run of
the norm, the step and the conversions together, as a training loop uses them.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import fsdp_sharded_optimizer_amd as zs
from tests import tensors_reference as ref
from tests.parity import from_np, to_np
from tests.test_gpu_tensors import same_bits

pytestmark = pytest.mark.gpu

SHAPES = [(33, 16), (16,), (70, 9), (1,), (300, 257), (128,)]
DECAY = [0.1, 0.0, 0.1, 0.0, 0.1, 0.0]       # none for the vectors


def start(dtype, seed=1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.rand(s, generator=gen, device="cuda") * 0.2 - 0.1).to(dtype) for s in SHAPES]


def gradients(t, dtype):
    gen = torch.Generator(device="cuda").manual_seed(100 + t)
    return [(torch.randn(s, generator=gen, device="cuda") * 0.05 * t).to(dtype) for s in SHAPES]


KW = dict(lr=3e-4, betas=(0.9, 0.95), weight_decay=DECAY, grad_scale=1 / 16, max_norm=1.0)


@pytest.mark.parametrize("pdtype,copy", [(torch.float32, True), (torch.float32, False), (torch.bfloat16, False)])
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
def test_five_steps_against_the_flat_calls(gdtype, pdtype, copy):
    """fp32 moments: the bits of the norm, then adamw_step (or _no_master) on
    each tensor by itself with its own decay."""
    params = start(pdtype)
    twin = [p.clone().reshape(-1) for p in params]
    copies = [torch.empty(p.shape, dtype=torch.bfloat16, device="cuda") for p in params] if copy else None
    tc = [torch.empty_like(p, dtype=torch.bfloat16) for p in twin]
    m, v = ([torch.zeros(p.numel(), device="cuda") for p in twin] for _ in range(2))
    opt = zs.TensorOptimizer(params, param_bf16=copies, **KW)
    norm = torch.zeros(1, dtype=torch.float64, device="cuda")
    for t in range(1, 6):
        gs = gradients(t, gdtype)
        opt.step(gs, extra_norm_sq=0.5)
        zs.grad_norm_sq_tensors(gs, 1 / 16, norm)
        assert opt.t == t and opt.norm_sq.item() == norm.item()
        for k, g in enumerate(gs):
            hp = zs.AdamWConfig(lr=3e-4, beta2=0.95, weight_decay=DECAY[k], grad_scale=1 / 16, max_norm=1.0,
                                extra_norm_sq=0.5, step=t)
            g = g.reshape(-1).float()
            if pdtype == torch.bfloat16:
                zs.adamw_step_no_master(hp, twin[k], m[k], v[k], g, norm_sq=norm)
            else:
                zs.adamw_step(hp, twin[k], m[k], v[k], g, tc[k] if copy else None, norm_sq=norm)
        for k, p in enumerate(params):
            assert same_bits(p.reshape(-1), twin[k]), (t, k)
            assert not copy or same_bits(copies[k].reshape(-1), tc[k])
        for got, want in zip(opt.moments(), (m, v)):
            assert all(same_bits(a, b) for a, b in zip(got, want)), t


def test_the_norm_clips_against_the_oracle():
    params = start(torch.float32)
    opt = zs.TensorOptimizer(params, **KW)
    gs = gradients(3, torch.float32)
    opt.step(gs)
    want = sum(oracle.grad_norm_sq(to_np(g.reshape(-1)), 1 / 16) for g in gs)
    # squares exact; under 1e5 additions of binary64
    assert abs(opt.norm_sq.item() - want) <= 1e5 * 2.0 ** -53 * want


@pytest.mark.parametrize("pdtype", [torch.float32, torch.bfloat16])
def test_8_bit_moments_follow_their_definition_over_a_run(pdtype):
    """Five steps: the stored moments bit for bit, parameters within their
    rounding (8 units of 2^-24 of u, as the step's own test; bf16 half a step)."""
    params = start(pdtype)
    opt = zs.TensorOptimizer(params, state_bits=8, seed=9, **KW)
    flat = [p.numel() for p in params]
    p64 = [to_np(p.reshape(-1).float()).astype(np.float64) for p in params]
    m, v = ([np.zeros(n, np.float32) for n in flat] for _ in range(2))
    groups = {0.1: [0, 2, 4], 0.0: [1, 3, 5]}
    for t in range(1, 6):
        gs = gradients(t, torch.bfloat16)
        opt.step(gs)
        coef = np.float32(min(1.0, 1.0 / (math.sqrt(opt.norm_sq.item()) + 1e-6)))
        for j, (decay, members) in enumerate(groups.items()):
            hp = zs.AdamWConfig(lr=3e-4, beta2=0.95, weight_decay=decay, grad_scale=1 / 16, max_norm=1.0, step=t)
            s, key = zs.adamw_scalars(hp), ref.key_of(9 + j, t)
            for index, k in enumerate(members):
                g = gs[k].reshape(-1).float().cpu().numpy()
                m[k], v[k] = ref.new_moments(g, m[k], v[k], s, coef)
                want, u = ref.update64(p64[k], m[k], v[k], s)
                m[k], v[k] = ref.stored(m[k], "m", index, key), ref.stored(v[k], "v", index, key)
                got = params[k].reshape(-1).float().cpu().numpy().astype(np.float64)
                bound = 2.0 ** -24 * (16 * np.abs(u) + 2 * np.abs(p64[k]) + np.abs(u))
                if pdtype == torch.bfloat16:
                    bound = bound + 2.0 ** -8 * np.abs(want)
                assert (np.abs(got - want) <= bound).all(), (t, k)
                p64[k] = got
        for got, want in zip(opt.moments(), (m, v)):
            assert all(np.array_equal(to_np(a).view(np.uint32), b.view(np.uint32)) for a, b in zip(got, want)), t


@pytest.mark.parametrize("bits", [32, 8])
def test_resume_is_bit_identical(bits):
    whole, parts = start(torch.float32), start(torch.float32)
    opt = zs.TensorOptimizer(whole, state_bits=bits, **KW)
    for t in range(1, 6):
        opt.step(gradients(t, torch.bfloat16))
    first = zs.TensorOptimizer(parts, state_bits=bits, **KW)
    for t in (1, 2):
        first.step(gradients(t, torch.bfloat16))
    saved = {k: x if k == "step" else [y.cpu() for y in x] for k, x in first.state_dict().items()}
    again = zs.TensorOptimizer(parts, state_bits=bits, **KW)
    again.load_state_dict(saved)
    for t in (3, 4, 5):
        again.step(gradients(t, torch.bfloat16))
    assert again.t == 5
    assert all(same_bits(a, b) for a, b in zip(whole, parts))
    for a, b in zip(opt.moments(), again.moments()):
        assert all(same_bits(x, y) for x, y in zip(a, b))


def test_the_widths_take_each_other_s_state():
    a = zs.TensorOptimizer(start(torch.float32), **KW)
    a.step(gradients(1, torch.float32))
    b = zs.TensorOptimizer([p.clone() for p in a.params], state_bits=8, **KW)
    b.load_state_dict(a.state_dict())
    for x, y in zip(a.moments()[1], b.moments()[1]):
        # one step of 3 fraction bits: at most 1/8 of the value
        assert ((x - y).abs() <= x / 8 + x.max() * 2.0 ** -33).all()
    c = zs.TensorOptimizer([p.clone() for p in a.params], **KW)
    c.load_state_dict(b.state_dict())
    assert all(same_bits(x, y) for x, y in zip(b.moments()[0], c.moments()[0]))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_is_the_eager_step(bits):
    params, twin = start(torch.float32), start(torch.float32)
    copies = [torch.empty(p.shape, dtype=torch.bfloat16, device="cuda") for p in params]
    opt = zs.TensorOptimizer(params, param_bf16=copies, state_bits=bits, seed=3, **KW)
    eager = zs.TensorOptimizer(twin, state_bits=bits, seed=3, **KW)
    grads = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in SHAPES]
    with pytest.raises(RuntimeError):
        opt.capture()
    opt.bind_grads(grads)
    opt.step(gradients(1, torch.bfloat16))
    eager.step(gradients(1, torch.bfloat16))
    opt.bind_grads(grads)
    graph = opt.capture(extra_norm_sq=0.25)
    assert opt.t == 1 and all(same_bits(a, b) for a, b in zip(params, twin))
    opt.bind_grads([torch.ones_like(g) for g in grads])      # the graph keeps the gradients it was captured on
    for t in range(2, 7):
        gs = gradients(t, torch.bfloat16)
        for to, g in zip(grads, gs):
            to.copy_(g)
        graph.replay()
        eager.step(gs, extra_norm_sq=0.25)
        torch.cuda.synchronize()
        assert opt.t == t
        assert all(same_bits(a, b) for a, b in zip(params, twin)), t
        for a, b in zip(opt.moments(), eager.moments()):
            assert all(same_bits(x, y) for x, y in zip(a, b)), t
        assert all(same_bits(c, p.to(torch.bfloat16)) for c, p in zip(copies, params))


def test_parameters_of_a_module_and_autograd_gradients():
    """nn.Parameters stepped on their .grad; a loss's gradients as autograd
    leaves them, new tensors every time."""
    torch.manual_seed(0)
    layer = torch.nn.Linear(40, 24, device="cuda")
    x = torch.randn(8, 40, device="cuda")
    for bits in (32, 8):
        opt = zs.TensorOptimizer(list(layer.parameters()), lr=1e-2, state_bits=bits)
        twin = [p.detach().clone() for p in layer.parameters()]
        layer.zero_grad(set_to_none=True)
        layer(x).square().mean().backward()
        grads = [p.grad for p in layer.parameters()]
        opt.step(grads)
        for p, q, g in zip(layer.parameters(), twin, grads):
            # a first step moves each parameter by lr * g / (|g| + eps)
            want = q.double() - 1e-2 * g.double() / (g.double().abs() + 1e-8)
            # u = lr and its roundings; the scalars' own (bias corrections of 1 - beta) to 2^-24 each, 1/(1-beta2) = 1000
            assert ((p.detach().double() - want).abs() <= 1e-2 * 64 * 2.0 ** -24 + 2.0 ** -23 * q.abs()).all()


def test_refusals():
    p = start(torch.float32)
    for bad in (dict(state_bits=16), dict(weight_decay=[0.1]), dict(seed=-1), dict(param_bf16=[None])):
        with pytest.raises(ValueError):
            zs.TensorOptimizer(p, lr=1e-3, **bad)
    with pytest.raises(ValueError):
        zs.TensorOptimizer([], lr=1e-3)
    with pytest.raises(TypeError):
        zs.TensorOptimizer([p[0].half()], lr=1e-3)
    with pytest.raises(ValueError):
        zs.TensorOptimizer([p[0].t()], lr=1e-3)
    with pytest.raises(ValueError):
        zs.TensorOptimizer([p[0].cpu()], lr=1e-3)
    opt = zs.TensorOptimizer(p, lr=1e-3)
    with pytest.raises(RuntimeError):
        opt.step()
    with pytest.raises(ValueError):
        opt.step(gradients(1, torch.float32)[:-1])
    before = [x.clone() for x in p]
    with pytest.raises(ValueError):
        opt.load_state_dict({"step": 1, "exp_avg": [torch.zeros(3)] * len(p), "exp_avg_sq": [torch.zeros(3)] * len(p)})
    assert opt.t == 0 and all(same_bits(a, b) for a, b in zip(before, p))


def test_moments_sit_where_the_step_is_aligned():
    """Parameters as views at odd offsets of one flat buffer: the fp32 moments
    start at the same offset from a cache line."""
    flat = torch.zeros(5000, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        flat = torch.zeros(5000, device="cuda", dtype=dtype)
        views = [flat[1:1000], flat[1000:1033], flat[1033:4999]]
        opt = zs.TensorOptimizer(views, lr=1e-3)
        for p, m, v in zip(views, *opt.moments()):
            lane = p.data_ptr() // p.element_size() % 32
            assert m.data_ptr() // 4 % 32 == lane and v.data_ptr() // 4 % 32 == lane


def test_no_step_is_half_refused():
    """What one of a step's calls would refuse, or could not see, is refused
    before the first: a bad decay, the same memory under two decays, a gradient
    in a parameter that another call writes, clipping without the norm."""
    p = start(torch.float32)
    for bad in (-0.1, math.nan, math.inf):
        with pytest.raises(ValueError):
            zs.TensorOptimizer(p, lr=1e-3, weight_decay=[0.1, bad] + [0.1] * 4)
    with pytest.raises(ValueError):
        zs.TensorOptimizer([p[0], p[0]], lr=1e-3, weight_decay=[0.1, 0.0])
    with pytest.raises(ValueError):
        zs.TensorOptimizer([p[0], p[0].reshape(-1)[-1:]], lr=1e-3, weight_decay=[0.1, 0.0])
    copy = p[1].view(torch.bfloat16).reshape(-1)[:16]
    with pytest.raises(ValueError):
        zs.TensorOptimizer(p[:2], lr=1e-3, weight_decay=[0.1, 0.0], param_bf16=[None, copy])
    with pytest.raises(ValueError):
        zs.TensorOptimizer(p, lr=1e-3, max_norm=1.0, compute_norm=False)
    empty = torch.empty(0, device="cuda")
    opt = zs.TensorOptimizer(p + [empty], lr=1e-3, weight_decay=DECAY + [0.0])
    grads = gradients(1, torch.float32) + [empty]
    before = [x.clone() for x in p]
    for k in range(len(p)):   # the parameter of another call, whole or only its last element
        with pytest.raises(ValueError):
            opt.step(grads[:k] + [p[k]] + grads[k + 1:])
    with pytest.raises(ValueError):
        opt.step(grads[:3] + [p[0].reshape(-1)[-1:]] + grads[4:])
    opt.max_norm = 1.0
    with pytest.raises(ValueError):
        opt.step(grads)
    assert opt.t == 0 and all(same_bits(a, b) for a, b in zip(before, p))
    opt.max_norm = 0.0
    # neighbours that only touch, and one gradient for two parameters, are fine
    flat = torch.zeros(200, device="cuda")
    g = torch.ones(100, device="cuda")
    opt = zs.TensorOptimizer([flat[:100], flat[100:]], lr=1e-3, weight_decay=[0.1, 0.0])
    opt.step([g, g])
    assert opt.t == 1 and bool((flat < 0).all()) and same_bits(flat[:100], flat[100:])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_follows_the_optimizer_or_refuses(bits):
    """lr, betas and max_norm may change between replays; what is recorded in
    the launches may not.  Capturing leaves every byte alone, also without a norm."""
    kw = dict(KW, state_bits=bits)
    params, twin = start(torch.float32), start(torch.float32)
    opt, eager = zs.TensorOptimizer(params, **kw), zs.TensorOptimizer(twin, **kw)
    grads = [g.clone() for g in gradients(3, torch.float32)]
    opt.step(grads)
    eager.step(grads)
    before = [x.clone() for x in (opt._states if bits == 8 else opt._exp_avg + opt._exp_avg_sq)]
    graph = opt.capture()
    for a, b in zip(before, opt._states if bits == 8 else opt._exp_avg + opt._exp_avg_sq):
        assert same_bits(a, b)
    assert all(same_bits(a, b) for a, b in zip(params, twin))
    for lr, betas, max_norm in ((1e-3, (0.9, 0.95), 1.0), (2e-3, (0.8, 0.99), 0.25), (5e-4, (0.9, 0.999), 0.0)):
        for o in (opt, eager):
            o.lr, o.betas, o.max_norm = lr, betas, max_norm
        graph.replay()
        eager.step()
        torch.cuda.synchronize()
        assert all(same_bits(a, b) for a, b in zip(params, twin)), (lr, betas, max_norm)
    t = opt.t
    for name, value in (("grad_scale", 1.0), ("compute_norm", False)):
        was = getattr(opt, name)
        setattr(opt, name, value)
        with pytest.raises(RuntimeError):
            graph.replay()
        setattr(opt, name, was)
    graph.replay()
    eager.step()
    torch.cuda.synchronize()
    assert opt.t == t + 1 and all(same_bits(a, b) for a, b in zip(params, twin))
    plain = zs.TensorOptimizer(params, lr=1e-3, state_bits=bits)
    plain.bind_grads(grads)
    graph = plain.capture()
    assert plain.t == 0 and all(same_bits(a, b) for a, b in zip(params, twin))
    plain.max_norm = 1.0
    with pytest.raises(ValueError):
        graph.replay()


def test_the_state_s_layout():
    """Moments at their parameters' offsets from a boundary of 256 elements,
    neighbours kept next to one another; 8-bit moments on boundaries of 1 KiB;
    nothing overlaps."""
    flat = torch.zeros(9000, device="cuda")
    params = [flat[3:1000], flat[1000:1001], flat[1001:5000], flat[6000:6300].clone(), torch.zeros(0, device="cuda"),
              flat[7001:8999]]
    opt = zs.TensorOptimizer(params, lr=1e-3)
    for ts in opt.moments():
        ends = 0
        for p, t in zip(params, ts):
            if t.numel():
                assert t.data_ptr() // 4 % 256 == p.data_ptr() // 4 % 256 and t.data_ptr() >= ends
                ends = t.data_ptr() + 4 * t.numel()
        assert ts[1].data_ptr() == ts[0].data_ptr() + 4 * 997 and ts[2].data_ptr() == ts[1].data_ptr() + 4
        assert all(not t.any() for t in ts)
    opt = zs.TensorOptimizer(params, lr=1e-3, state_bits=8)
    ends = 0
    for p, s in zip(params, opt._states):
        assert s.numel() == zs.moments_q8_bytes(p.numel())
        if s.numel():
            assert s.data_ptr() % 1024 == 0 and s.data_ptr() >= ends
            ends = s.data_ptr() + s.numel()
