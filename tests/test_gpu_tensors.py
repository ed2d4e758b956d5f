"""The gradient norm and AdamW (fp32 moments) over lists of tensors on the GPU.

Sizes from one element up, around the vector, tile and table lengths, empty
tensors, more tensors than one launch takes, and views at odd offsets; every
buffer lies between guard values that must stay.  The update is compared bit
for bit with adamw_step / adamw_step_no_master of each tensor, and with the
formula in binary64.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import fsdp_sharded_optimizer_amd as zs
from tests import tensors_reference as ref
from tests.parity import bits_equal, from_np, to_np

pytestmark = pytest.mark.gpu

LISTS = {
    "one": [1],
    "edges": [1, 2, 3, 4, 5, 63, 64, 255, 256, 257, 0, 511, 1023, 1024, 1025],
    "many": [(37 * k) % 700 for k in range(250)],          # zeros among them; three launches, two for the norm
    "one table": [256] * 98,
    "a table and one": [300] * 99,
    "large": [1_000_003, 7, 262_144],
}
GUARD = 17        # elements on each side


class Pool:
    """Tensors of one dtype as views of one buffer with guards between them:
    each on a 512-byte boundary, or back to back behind `odd` elements."""

    def __init__(self, numels, dtype, packed=None, fill=None):
        self.views, at = [], 0
        spots = []
        for n in numels:
            at += GUARD
            if packed is None:
                at = -(-at // 256) * 256
            elif not spots:
                at += packed
            spots.append(at)
            at += n
        self.buffer = torch.full((at + GUARD,), 7.75, dtype=dtype, device="cuda")
        self.views = [self.buffer[a:a + n] for a, n in zip(spots, numels)]
        self.inside = torch.zeros(at + GUARD, dtype=torch.bool, device="cuda")
        for a, n in zip(spots, numels):
            self.inside[a:a + n] = True
        if fill is not None:
            for v, x in zip(self.views, fill):
                v.copy_(from_np(x) if isinstance(x, np.ndarray) else x)

    def guards_stand(self):
        return bool((self.buffer[~self.inside] == 7.75).all())


def draws(numels, seed, std, cast=False):
    rng = np.random.default_rng(seed)
    out = [(rng.standard_normal(n) * std).astype(np.float32) for n in numels]
    return [oracle.bf16_widen(oracle.bf16_rne(x)) for x in out] if cast else out


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [None, 0, 1])
@pytest.mark.parametrize("name", LISTS)
def test_norm(name, packed, dtype):
    print(name, packed, dtype, flush=True)
    numels = LISTS[name]
    gs = draws(numels, 3, 1e-2, dtype == torch.bfloat16)
    pool = Pool(numels, dtype, packed, gs)
    out = torch.full((2,), -1.0, dtype=torch.float64, device="cuda")
    lst = zs.GradTensors(pool.views)
    need = zs.grad_norm_sq_tensors_workspace_bytes(lst)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    for scale in (1 / 64, 0.3):
        zs.grad_norm_sq_tensors(lst, scale, out[:1], ws[:need])
        want = math.fsum(math.fsum((x * np.float32(scale)).astype(np.float64) ** 2) for x in gs)
        got = out[0].item()
        # squares exact; at most N additions, each off by half a binary64 step of at most the total
        assert abs(got - want) <= sum(numels) * 2.0 ** -53 * want
        zs.grad_norm_sq_tensors(pool.views, scale, out[:1])                 # the same bits from a plain list
        assert out[0].item() == got and out[1].item() == -1.0
    assert (ws[need:] == 0xA5).all() and pool.guards_stand()


def test_norm_of_nothing_and_of_non_finite_values():
    out = torch.full((1,), 5.0, dtype=torch.float64, device="cuda")
    zs.grad_norm_sq_tensors([], 1.0, out)
    assert out.item() == 0.0
    out.fill_(5.0)
    zs.grad_norm_sq_tensors([torch.empty(0, device="cuda")], 1.0, out)
    assert out.item() == 0.0
    for bad in (math.inf, -math.inf, math.nan):
        g = torch.zeros(5000, device="cuda")
        g[4999] = bad
        zs.grad_norm_sq_tensors([torch.ones(10, device="cuda"), g], 1.0, out)
        assert not math.isfinite(out.item())
    g = torch.ones(3, device="cuda")
    zs.grad_norm_sq_tensors([g, g, g], 1.0, out)                            # one gradient three times
    assert out.item() == 9.0


def test_norm_does_not_depend_on_alignment():
    numels = LISTS["edges"] + [20_001]
    gs = draws(numels, 4, 1.0, True)
    got = set()
    for packed in (None, 0, 1, 2, 5):
        out = torch.zeros(1, dtype=torch.float64, device="cuda")
        zs.grad_norm_sq_tensors(Pool(numels, torch.bfloat16, packed, gs).views, 0.3, out)
        got.add(out.item())
    assert len(got) == 1


HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, grad_scale=1 / 64)


def a_list(numels, pdtype, gdtype, copy, packed, seed=5):
    """Pools of params, grads, moments and re-casts, and their start in numpy."""
    p = draws(numels, seed, 0.05, pdtype == torch.bfloat16)
    g = draws(numels, seed + 1, 0.1, gdtype == torch.bfloat16)
    m = draws(numels, seed + 2, 1e-4)
    v = [np.abs(x) for x in draws(numels, seed + 3, 1e-6)]
    pools = {"p": Pool(numels, pdtype, packed, p), "g": Pool(numels, gdtype, packed, g),
             "m": Pool(numels, torch.float32, packed, m), "v": Pool(numels, torch.float32, packed, v)}
    if copy:
        pools["c"] = Pool(numels, torch.bfloat16, packed)
    return pools, p, g, m, v


def adamw_list(pools):
    return zs.AdamWTensors(pools["p"].views, pools["g"].views, pools["m"].views, pools["v"].views,
                           pools["c"].views if "c" in pools else None)


def one_by_one(pools, hp, norm):
    """The flat step of each tensor on copies (its gradient widened)."""
    out = []
    for k, p in enumerate(pools["p"].views):
        p, m, v = p.clone(), pools["m"].views[k].clone(), pools["v"].views[k].clone()
        g = pools["g"].views[k].float()
        c = torch.zeros(p.numel(), dtype=torch.bfloat16, device="cuda") if "c" in pools else None
        if p.dtype == torch.bfloat16:
            zs.adamw_step_no_master(hp, p, m, v, g, norm_sq=norm)
        else:
            zs.adamw_step(hp, p, m, v, g, c, norm_sq=norm)
        out.append({"p": p, "m": m, "v": v, "c": c})
    return out


def same_bits(a, b):
    return bits_equal(to_np(a), to_np(b))


@pytest.mark.parametrize("pdtype,copy", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [None, 0, 1, 3])
@pytest.mark.parametrize("name", LISTS)
def test_step_is_the_flat_step_of_each_tensor(name, packed, gdtype, pdtype, copy):
    print(name, packed, gdtype, pdtype, copy, flush=True)
    pools, *_ = a_list(LISTS[name], pdtype, gdtype, copy, packed)
    lst = adamw_list(pools)
    norm = torch.tensor([2.5], dtype=torch.float64, device="cuda")
    for t, clip in ((1, 0.0), (2, 1.0), (3, 100.0)):
        hp = zs.AdamWConfig(**HP, max_norm=clip, step=t)
        want = one_by_one(pools, hp, norm if clip else None)
        zs.adamw_step_tensors(hp, lst, norm_sq=norm if clip else None)
        for k, w in enumerate(want):
            for name_ in ("p", "m", "v") + (("c",) if copy else ()):
                assert same_bits(pools[name_].views[k], w[name_]), (t, k, name_)
    assert all(pool.guards_stand() for pool in pools.values())


@pytest.mark.parametrize("pdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
def test_step_against_the_formula_in_64_bits(gdtype, pdtype):
    """u: 4 roundings each of the moments' inputs, root, quotient, sum, ratio and
    product: below 12 * 2^-24 of |u|; the parameter's product and difference
    2^-24 of |p| each; bf16 half a step, 2^-8, of the result."""
    numels = [1, 5, 1000, 4097]
    pools, p, g, m, v = a_list(numels, pdtype, gdtype, False, None)
    t, S, clip = 4, 9.0, 1.5
    zs.adamw_step_tensors(zs.AdamWConfig(**HP, max_norm=clip, step=t), adamw_list(pools),
                          norm_sq=torch.tensor([S], dtype=torch.float64, device="cuda"))
    coef = min(1.0, clip / (math.sqrt(S) + 1e-6))
    e24 = 2.0 ** -24
    for k in range(len(numels)):
        gg = g[k].astype(np.float64) / 64 * coef
        mm = 0.9 * m[k].astype(np.float64) + 0.1 * gg
        vv = 0.95 * v[k].astype(np.float64) + 0.05 * gg * gg
        u = HP["lr"] / (1 - 0.9 ** t) * mm / (np.sqrt(vv) / math.sqrt(1 - 0.95 ** t) + 1e-8)
        pp = p[k].astype(np.float64) * (1 - HP["lr"] * HP["weight_decay"]) - u
        # the scalars and coef are rounded (2 of 2^-24 each term), each sum may cancel: relative to its terms
        terms = 0.9 * np.abs(m[k]) + 0.1 * np.abs(gg)
        assert (np.abs(pools["m"].views[k].cpu().double().numpy() - mm) <= 6 * e24 * terms).all()
        assert (np.abs(pools["v"].views[k].cpu().double().numpy() - vv) <= 10 * e24 * vv).all()
        du = HP["lr"] / (1 - 0.9 ** t) * terms / (np.sqrt(vv) / math.sqrt(1 - 0.95 ** t) + 1e-8)
        bound = 20 * e24 * du + 3 * e24 * np.abs(p[k])
        if pdtype == torch.bfloat16:
            bound = bound + 2.0 ** -8 * np.abs(pp)
        assert (np.abs(pools["p"].views[k].cpu().double().numpy() - pp) <= bound).all()


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_a_non_finite_norm_leaves_everything(bad):
    pools, *_ = a_list(LISTS["edges"], torch.float32, torch.bfloat16, True, 1)
    before = {k: pool.buffer.clone() for k, pool in pools.items()}
    zs.adamw_step_tensors(zs.AdamWConfig(**HP, max_norm=1.0), adamw_list(pools),
                          norm_sq=torch.tensor([bad], dtype=torch.float64, device="cuda"))
    for k, x in before.items():
        assert same_bits(pools[k].buffer, x), k


def test_mixed_streams_offsets_and_missing_copies():
    """Each stream at an offset of its own, re-casts for some tensors only, and
    a gradient shared by two tensors."""
    numels = [1000, 515, 77, 4096]
    pools, *_ = a_list(numels, torch.float32, torch.float32, True, None)
    pools["p"] = Pool(numels, torch.float32, 1, [x.clone() for x in pools["p"].views])
    pools["m"] = Pool(numels, torch.float32, 2, [x.clone() for x in pools["m"].views])
    g = pools["g"].views
    g[3].copy_(torch.cat([g[0], g[0], g[0], g[0], torch.zeros(96, device="cuda")]))
    shared = [g[3][:1000], g[1], g[2], g[3]]                # tensor 0's gradient is a part of tensor 3's
    copies = [pools["c"].views[0], None, pools["c"].views[2], None]
    hp = zs.AdamWConfig(**HP, step=2)
    pools["g"].views = shared
    want = one_by_one(pools, hp, None)
    untouched = [pools["c"].views[k].clone() for k in (1, 3)]
    zs.adamw_step_tensors(hp, zs.AdamWTensors(pools["p"].views, shared, pools["m"].views, pools["v"].views, copies))
    for k, w in enumerate(want):
        for n in ("p", "m", "v"):
            assert same_bits(pools[n].views[k], w[n]), (k, n)
        if copies[k] is not None:
            assert same_bits(copies[k], w["c"])
    assert same_bits(pools["c"].views[1], untouched[0]) and same_bits(pools["c"].views[3], untouched[1])


def test_set_grads_and_refusals():
    p = torch.zeros(8, device="cuda")
    lst = zs.AdamWTensors([p], [torch.ones(8, device="cuda")], [p.clone()], [p.clone()])
    hp = zs.AdamWConfig(lr=1.0, step=1)
    zs.adamw_step_tensors(hp, lst)
    assert torch.allclose(p, torch.full_like(p, -1.0))
    lst.set_grads([torch.full((8,), -1.0, dtype=torch.bfloat16, device="cuda")])
    zs.adamw_step_tensors(hp, lst)
    assert lst.grad_dtype == 1 and torch.isfinite(p).all()
    with pytest.raises(ValueError):
        lst.set_grads([torch.ones(7, device="cuda")])
    with pytest.raises(TypeError):
        lst.set_grads([torch.ones(8, device="cuda", dtype=torch.float16)])
    with pytest.raises(ValueError):
        lst.set_grads([torch.ones(8, 2, device="cuda")[:, 0]])             # not contiguous
    with pytest.raises(ValueError):
        lst.set_grads([])
    b = torch.zeros(8, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        zs.AdamWTensors([b], [p], [p.clone()], [p.clone()], [b.clone()])   # a re-cast of bf16 parameters
    with pytest.raises(TypeError):
        zs.AdamWTensors([p, b], [p, p], [p, p], [p, p])                    # two dtypes
    with pytest.raises(zs.ZShardError):
        zs.adamw_step_tensors(hp, zs.AdamWTensors([p], [p], [p.clone()], [p.clone()]))


def test_dev_scalars_and_a_captured_graph():
    """The norm and the step captured once, replayed for later steps with new
    gradients and scalars: each replay is the eager step, also with eager work
    of other lists in between."""
    numels = LISTS["many"] + [50_001]
    pools, *_ = a_list(numels, torch.float32, torch.bfloat16, True, 1)
    twin = {k: Pool(numels, pool.buffer.dtype, 1, [v.clone() for v in pool.views]) for k, pool in pools.items()}
    lst, eager = adamw_list(pools), adamw_list(twin)
    grads, egrads = zs.GradTensors(pools["g"].views), zs.GradTensors(twin["g"].views)
    need = zs.grad_norm_sq_tensors_workspace_bytes(grads)
    norm, enorm = (torch.zeros(1, dtype=torch.float64, device="cuda") for _ in range(2))
    ws, ews = (torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(2))
    sc = torch.zeros(56, dtype=torch.uint8, device="cuda")

    def body():
        zs.grad_norm_sq_tensors(grads, 1 / 64, norm, ws)
        zs.adamw_step_tensors_dev(sc, lst, norm_sq=norm)

    def scalars(t):
        hp = zs.AdamWConfig(**HP, max_norm=0.5, step=t)
        sc.copy_(torch.frombuffer(bytearray(zs.scalars_bytes(hp)), dtype=torch.uint8))
        return hp
    saved = {k: pool.buffer.clone() for k, pool in pools.items()}
    scalars(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for k, x in saved.items():
        pools[k].buffer.copy_(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for t in range(1, 5):
        for k, x in enumerate(draws(numels, 50 + t, 0.05 * t, True)):
            pools["g"].views[k].copy_(from_np(x))
            twin["g"].views[k].copy_(from_np(x))
        hp = scalars(t)
        graph.replay()
        zs.grad_norm_sq_tensors(egrads, 1 / 64, enorm, ews)
        zs.adamw_step_tensors(hp, eager, norm_sq=enorm)
        torch.cuda.synchronize()
        assert norm.item() == enorm.item()
        for k in ("p", "m", "v", "c"):
            assert same_bits(pools[k].buffer, twin[k].buffer), (t, k)


def test_two_streams_and_two_lists_at_once():
    lists = []
    for seed in (5, 25):
        pools, *_ = a_list(LISTS["large"], torch.float32, torch.bfloat16, True, None, seed)
        lists.append(pools)
    hp = [zs.AdamWConfig(**HP, step=t) for t in (1, 2, 3)]
    want = [[one_by_one(pools, hp[0], None)] for pools in lists]
    streams = [torch.cuda.Stream() for _ in lists]
    torch.cuda.synchronize()
    for pools, stream in zip(lists, streams):
        zs.adamw_step_tensors(hp[0], adamw_list(pools), stream=stream)
    torch.cuda.synchronize()
    for pools, w in zip(lists, want):
        for k in range(len(LISTS["large"])):
            assert same_bits(pools["p"].views[k], w[0][k]["p"])


def test_offsets_past_32_bits():
    """A tensor of more than 2^31 elements behind a small one (bf16 parameters):
    elements on both sides of each 2^31 boundary and the last ones."""
    n = (1 << 31) + 1001
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    small = [torch.ones(5, dtype=d, device="cuda") for d in (torch.bfloat16, torch.bfloat16, torch.float32, torch.float32)]
    spots = [0, 1, 255, 256, (1 << 30) - 1, 1 << 30, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, n - 2, n - 1]
    for k, at in enumerate(spots):
        g[at] = k + 1.0
        p[at] = 2.0
    lst = zs.AdamWTensors([small[0], p], [small[1], g], [small[2], m], [small[3], v])
    norm = torch.zeros(1, dtype=torch.float64, device="cuda")
    zs.grad_norm_sq_tensors([small[1], g], 1.0, norm)
    assert norm.item() == 5 + sum((k + 1.0) ** 2 for k in range(len(spots)))
    zs.adamw_step_tensors(zs.AdamWConfig(lr=0.5, beta1=0.5, beta2=0.75), lst)
    got_m, got_v = m[spots].cpu(), v[spots].cpu()
    assert got_m.tolist() == [0.5 * (k + 1) for k in range(len(spots))]
    assert got_v.tolist() == [0.25 * (k + 1) ** 2 for k in range(len(spots))]
    assert (p[spots].cpu().float() - 1.5).abs().max() <= 2.0 ** -8 * 1.5
    assert int(torch.count_nonzero(m)) == len(spots) and int(torch.count_nonzero(p)) == len(spots)


def test_the_norm_s_own_workspace_on_another_stream():
    """Without a workspace the call takes one of the stream it runs on: memory
    that is freed when it returns, while the kernels have yet to run, is not
    handed to the current stream."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    grads = [torch.randn(300_000, generator=gen, device="cuda") for _ in range(4)]
    lst = zs.GradTensors(grads)
    need = zs.grad_norm_sq_tensors_workspace_bytes(lst)
    want = zs.grad_norm_sq_tensors(lst, 1.0, torch.zeros(1, dtype=torch.float64, device="cuda"))
    slow = torch.randn(4096, 4096, generator=gen, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = torch.zeros(1, dtype=torch.float64, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(4):
            slow @ slow
    zs.grad_norm_sq_tensors(lst, 1.0, out, stream=side)
    taken = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert same_bits(out, want) and all(bool((t == 255).all()) for t in taken)


@pytest.mark.parametrize("broken", [None, "p", "g", "m", "v", "c", "missing", "order"])
def test_tensors_that_follow_one_another(broken):
    """Views of flat buffers, where neighbours may be taken as one, and lists in
    which one stream is not like that: moved at one tensor, without a re-cast,
    or with the tensors in another order."""
    numels = [300, 1, 0, 255, 1024, 77, 0, 513, 31]
    pools, *_ = a_list(numels, torch.float32, torch.bfloat16, True, 1)
    if broken in pools:     # the fifth tensor's is elsewhere
        x = pools[broken].views[4]
        pools[broken].views[4] = x.clone()
    copies = list(pools["c"].views)
    if broken == "missing":
        copies[3] = copies[4] = None
    order = list(range(len(numels)))
    if broken == "order":
        order = [1, 0, 2, 4, 3, 5, 8, 7, 6]
    hp = zs.AdamWConfig(**HP, step=3)
    want = one_by_one(pools, hp, None)
    pick = lambda ts: [ts[k] for k in order]  # noqa: E731
    left = [c.clone() for c in pools["c"].views]
    zs.adamw_step_tensors(hp, zs.AdamWTensors(pick(pools["p"].views), pick(pools["g"].views), pick(pools["m"].views),
                                              pick(pools["v"].views), pick(copies)))
    for k, w in enumerate(want):
        for n in ("p", "m", "v"):
            assert same_bits(pools[n].views[k], w[n]), (k, n)
        assert same_bits(pools["c"].views[k], w["c"] if copies[k] is not None else left[k]), k


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_around_a_tile_at_every_offset(dtype):
    """Lengths around the ends of tiles, at offsets of 0 to 8 elements, between
    values that are not numbers: the bits of the same tensor by itself."""
    for n in (1, 7, 8, 511, 512, 513, 4095, 4096, 4097, 8191, 8192, 8193, 16384, 16391, 24577):
        x = torch.from_numpy(draws([n], n, 1.0, dtype == torch.bfloat16)[0]).to("cuda", dtype)
        want = zs.grad_norm_sq_tensors([x], 0.3, torch.zeros(1, dtype=torch.float64, device="cuda"))
        for off in range(9):
            buffer = torch.full((n + 80,), math.nan, dtype=dtype, device="cuda")
            view = buffer[32 + off:32 + off + n]
            view.copy_(x)
            out = zs.grad_norm_sq_tensors([view], 0.3, torch.zeros(1, dtype=torch.float64, device="cuda"))
            assert same_bits(out, want), (n, off)


def at_offset(x, off):
    """A copy of x that starts `off` elements into a buffer."""
    buffer = torch.zeros(x.numel() + 64, dtype=x.dtype, device="cuda")
    buffer[off:off + x.numel()] = x
    return buffer[off:off + x.numel()]


@pytest.mark.parametrize("gdtype,n", [(torch.bfloat16, 130_000_003), (torch.float32, 65_000_001)])
def test_long_gradients_at_any_offset(gdtype, n):
    """More gradients than the last-level cache holds: norm and step of views
    at odd offsets against the same list on 512-byte boundaries."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    p, m, v, g = (torch.randn(n, generator=gen, device="cuda") * s for s in (0.05, 1e-3, 1e-3, 0.1))
    v, g = v * v, g.to(gdtype)
    hp = zs.AdamWConfig(**HP, max_norm=1.0, step=4)
    done = []
    for offs in ((0, 0, 0, 0, 0), (1, 1, 1, 1, 1), (0, 3, 1, 2, 5)):
        ps, gs, ms, vs = (at_offset(x, o) for x, o in zip((p, g, m, v), offs))
        c = at_offset(torch.zeros(n, dtype=torch.bfloat16, device="cuda"), offs[4])
        norm = zs.grad_norm_sq_tensors([gs], hp.grad_scale, torch.zeros(1, dtype=torch.float64, device="cuda"))
        zs.adamw_step_tensors(hp, zs.AdamWTensors([ps], [gs], [ms], [vs], [c]), norm_sq=norm)
        done.append((norm, ps, ms, vs, c))
        for a, b in zip(done[0], done[-1]):
            assert torch.equal(a, b), offs
        done[1:] = []


@pytest.mark.parametrize("gdtype,pdtype,copy", [(torch.float32, torch.float32, False), (torch.bfloat16, torch.float32, True),
                                                (torch.bfloat16, torch.bfloat16, False)])
def test_step_at_every_kind_of_offset(gdtype, pdtype, copy):
    """Streams at one offset from a tile, at two, and at offsets of their own;
    lengths around a tile."""
    for n in (1, 255, 256, 257, 600):
        pools, *_ = a_list([n], pdtype, gdtype, copy, None, seed=n)
        hp = zs.AdamWConfig(**HP, step=2)
        want = one_by_one(pools, hp, None)[0]
        for offs in ((0,) * 5, (1,) * 5, (31,) * 5, (128,) * 5, (255,) * 5, (0, 0, 255, 255, 0), (7, 0, 32, 64, 1),
                     (64, 3, 31, 32, 5)):
            names = "pgmvc" if copy else "pgmv"
            guarded = {}
            for name, off in zip(names, offs):
                x = pools[name].views[0]
                buffer = torch.full((n + 600,), 7.75, dtype=x.dtype, device="cuda")
                buffer[256 + off:256 + off + n] = x
                guarded[name] = buffer
            at = {name: b[256 + off:256 + off + n] for (name, b), off in zip(guarded.items(), offs)}
            zs.adamw_step_tensors(hp, zs.AdamWTensors([at["p"]], [at["g"]], [at["m"]], [at["v"]],
                                                      [at["c"]] if copy else None))
            for name, off in zip(names, offs):
                if name != "g":
                    assert same_bits(at[name], want[name]), (n, offs, name)
                b = guarded[name]
                assert bool((b[:256 + off] == 7.75).all()) and bool((b[256 + off + n:] == 7.75).all()), (n, offs, name)


@pytest.mark.parametrize("count", [255, 256, 257, 327, 328, 329, 656, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_norm_of_many_tensors(dtype, count):
    """Lists around what one table holds: empty tensors, one element, whole tiles
    and ragged ones among them."""
    tile = 8192 if dtype == torch.bfloat16 else 4096
    kinds = [1, 0, 17, tile, tile + 1, 300, 2 * tile - 1, 8]
    numels = [kinds[(k * k + k // 7) % 8] for k in range(count)]
    gs = draws(numels, count, 0.1, dtype == torch.bfloat16)
    want = math.fsum(math.fsum((x * np.float32(0.3)).astype(np.float64) ** 2) for x in gs)
    got = set()
    for packed in (None, 1):
        out = torch.zeros(1, dtype=torch.float64, device="cuda")
        zs.grad_norm_sq_tensors(Pool(numels, dtype, packed, gs).views, 0.3, out)
        got.add(out.item())
    assert len(got) == 1
    # squares exact; at most N additions, each off by half a binary64 step of at most the total
    assert abs(got.pop() - want) <= sum(numels) * 2.0 ** -53 * want


@pytest.mark.parametrize("parts", [1, 2, 2047, 2048, 2049, 4097, 16383, 16384, 16385, 40000])
def test_norm_s_partials(parts):
    """One tile per partial, by count around where their sum changes its launches:
    small whole numbers, whose squares add exactly."""
    n = parts * 4096 - 5
    x = torch.arange(n, device="cuda", dtype=torch.int32).remainder_(7).float()
    lst = zs.GradTensors([x[:n // 2], x[n // 2:]] if parts == 2 else [x])
    need = zs.grad_norm_sq_tensors_workspace_bytes(lst)
    ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    out = torch.zeros(1, dtype=torch.float64, device="cuda")
    for _ in range(2):
        zs.grad_norm_sq_tensors(lst, 1.0, out, ws[:need])
        whole, rest = divmod(n, 7)
        assert out.item() == whole * sum(k * k for k in range(7)) + sum(k * k for k in range(rest))
    assert bool((ws[need:] == 0xA5).all())
