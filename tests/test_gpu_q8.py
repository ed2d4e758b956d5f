"""8-bit moments on the GPU: the conversions and the AdamW step over lists.

Codes depend on the last bit of a moment, so what is stored is compared bit
for bit with the definition in numpy; the parameter with the formula in
binary64.
"""
import math

import numpy as np
import pytest
import torch

import oracle
import fsdp_sharded_optimizer_amd as zs
from tests import tensors_reference as ref
from tests.parity import from_np, to_np
from tests.test_gpu_tensors import HP, LISTS, Pool, at_offset, draws, same_bits

pytestmark = pytest.mark.gpu

E24 = 2.0 ** -24


def states_of(numels):
    """8-bit states with guard bytes behind each."""
    full = [torch.full((zs.moments_q8_bytes(n) + 128,), 0xA5, dtype=torch.uint8, device="cuda") for n in numels]
    return full, [x[:zs.moments_q8_bytes(n)] for x, n in zip(full, numels)]


def guards_stand(full):
    return all(bool((x[-128:] == 0xA5).all()) for x in full)


def moments_for(numels, seed, spread=0.0):
    rng = np.random.default_rng(seed)
    out = []
    for n in numels:
        scale = np.exp2(-rng.uniform(0, spread, n)) if spread else 1.0
        m = (rng.standard_normal(n) * 1e-4 * scale).astype(np.float32)
        out.append((m, ((rng.standard_normal(n) * 1e-3 * scale) ** 2).astype(np.float32)))
    return [a for a, _ in out], [b for _, b in out]


def decoded(states, numels, dtype=torch.float32, packed=None):
    m, v = Pool(numels, dtype, packed), Pool(numels, dtype, packed)
    zs.moments_q8_decode(zs.Q8Moments(states, m.views, v.views, numels))
    assert m.guards_stand() and v.guards_stand()
    return m.views, v.views


def equal_values(got, want):
    """Bit for bit, NaN for NaN."""
    a, b = got.cpu().float().numpy(), want
    nan = np.isnan(b)
    return np.array_equal(np.isnan(a), nan) and np.array_equal(a[~nan].view(np.uint32), b[~nan].view(np.uint32))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [None, 0, 1])
@pytest.mark.parametrize("name", LISTS)
def test_conversions(name, packed, dtype):
    print(name, packed, dtype, flush=True)
    numels = LISTS[name]
    m, v = moments_for(numels, 7, 20.0)
    pm, pv = Pool(numels, dtype, packed, m), Pool(numels, dtype, packed, v)
    m, v = ([x.cpu().float().numpy() for x in pool.views] for pool in (pm, pv))
    full, states = states_of(numels)
    key = ref.key_of(99, 0)
    zs.moments_q8_encode(zs.Q8Moments(states, pm.views, pv.views), seed=99)
    gm, gv = decoded(states, numels, dtype, packed)
    for k in range(len(numels)):
        assert equal_values(gm[k], ref.stored(m[k], "m", k, key)), k
        assert equal_values(gv[k], ref.stored(v[k], "v", k, key)), k
    assert guards_stand(full) and pm.guards_stand() and pv.guards_stand()
    # what was read out and is stored again keeps its values, whatever the seed
    _, again = states_of(numels)
    zs.moments_q8_encode(zs.Q8Moments(again, gm, gv), seed=3)
    am, av = decoded(again, numels, dtype)
    for k in range(len(numels)):
        assert same_bits(am[k], gm[k]) and same_bits(av[k], gv[k]), k


def test_conversion_edges():
    """Zeros, both zeros' signs, subnormals, the largest numbers, values at and
    over the top code, infinities and NaN (their block reads as NaN), a
    negative second moment (its magnitude)."""
    f = np.float32
    rows = [np.zeros(300, f), np.full(300, -0.0, f), np.full(256, 1e-44, f), np.full(10, 1.875, f),
            np.full(300, np.nextafter(f(1.875), f(2)), f), np.full(256, 3.1e38, f), np.full(256, 3.3e38, f)]
    for bad in (np.inf, -np.inf, np.nan, np.uint32(0x7FFFFFFF).view(f), np.uint32(0xFFFFFFFF).view(f)):
        x = np.ones(600, f)
        x[299] = bad
        rows.append(x)
    x = np.linspace(-1, 1, 700).astype(f)
    rows += [x, x * f(1e-38), x * f(2.0 ** -149 / 1e-3), np.geomspace(1e-45, 1e30, 256).astype(f)]
    numels = [r.size for r in rows]
    full, states = states_of(numels)
    src = [from_np(r) for r in rows]
    zs.moments_q8_encode(zs.Q8Moments(states, src, [s.clone() for s in src]), seed=1)
    gm, gv = decoded(states, numels)
    key = ref.key_of(1, 0)
    for k, r in enumerate(rows):
        assert equal_values(gm[k], ref.stored(r, "m", k, key)), k
        assert equal_values(gv[k], ref.stored(np.abs(r), "v", k, key)), k
    assert guards_stand(full)


def test_the_largest_values():
    """Around 1.875 * 2^127: blocks of that value alone, and with it negative beside small ones."""
    rows = []
    for bits in (0x7F6FFFFF, 0x7F700000, 0x7F700001):
        top = np.uint32(bits).view(np.float32)
        row = np.linspace(0.25, 1, 300).astype(np.float32)
        row[7] = -top
        rows += [np.full(256, top), row]
    numels = [r.size for r in rows]
    full, states = states_of(numels)
    zs.moments_q8_encode(zs.Q8Moments(states, [from_np(r) for r in rows], [from_np(np.abs(r)) for r in rows]), seed=3)
    gm, gv = decoded(states, numels)
    key = ref.key_of(3, 0)
    for k, r in enumerate(rows):
        assert equal_values(gm[k], ref.stored(r, "m", k, key)), k
        assert equal_values(gv[k], ref.stored(np.abs(r), "v", k, key)), k
        assert bool(torch.isnan(gm[k][:256]).all()) == (k >= 4) and not torch.isnan(gm[k][256:]).any()
    assert bool((gm[2] == rows[2][0]).all()) and bool((gv[2] == rows[2][0]).all())      # kept as it is
    assert guards_stand(full)


def test_bf16_holds_the_values_from_2_to_the_minus_130():
    """Read out into bf16: the values that fp32 holds, exactly from 2^-130 up and
    to nearest below it (bf16's least step is 2^-133); stored again, the same."""
    rng = np.random.default_rng(12)
    rows = [(np.exp2(rng.uniform(lo, lo + 12, 512)) * (1 if lo % 2 else -1)).astype(np.float32)
            for lo in (-149, -144, -138, -135, -132, -131, -130, -126)]
    numels = [r.size for r in rows]
    _, states = states_of(numels)
    zs.moments_q8_encode(zs.Q8Moments(states, [from_np(r) for r in rows], [from_np(np.abs(r)) for r in rows]), seed=5)
    wide, narrow = decoded(states, numels), decoded(states, numels, torch.bfloat16)
    inexact = 0
    for w, b in zip(wide[0] + wide[1], narrow[0] + narrow[1]):
        w, b = w.cpu().numpy(), b.cpu().float().numpy()
        assert np.array_equal(oracle.bf16_widen(oracle.bf16_rne(w)).view(np.uint32), b.view(np.uint32))
        large = np.abs(w) >= 2.0 ** -130
        assert np.array_equal(w[large], b[large])
        inexact += int((w != b).sum())
    assert inexact > 0
    _, again = states_of(numels)
    zs.moments_q8_encode(zs.Q8Moments(again, *narrow), seed=6)
    for x, y in zip(narrow[0] + narrow[1], sum(decoded(again, numels, torch.bfloat16), [])):
        assert same_bits(x, y)


def test_missing_moments_and_a_fresh_state():
    numels = [5, 1000]
    zero = [torch.zeros(zs.moments_q8_bytes(n), dtype=torch.uint8, device="cuda") for n in numels]
    gm, gv = decoded(zero, numels)
    assert all(not x.any() for x in gm + gv)                 # zero bytes hold zero moments
    m, v = moments_for(numels, 8)
    _, states = states_of(numels)
    zs.moments_q8_encode(zs.Q8Moments(states, None, [from_np(x) for x in v]), seed=2)
    gm, gv = decoded(states, numels)
    key = ref.key_of(2, 0)
    for k in range(2):
        assert not gm[k].any() and equal_values(gv[k], ref.stored(v[k], "v", k, key))
    out = torch.full((1000,), 3.0, device="cuda")
    zs.moments_q8_decode(zs.Q8Moments(states, None, [None, out], numels))   # the first tensor is skipped
    assert equal_values(out, ref.stored(v[1], "v", 1, key))


def make(numels, pdtype, gdtype, copy, packed, seed=31, spread=0.0):
    p = draws(numels, seed, 0.05, pdtype == torch.bfloat16)
    g = draws(numels, seed + 1, 0.1, gdtype == torch.bfloat16)
    m, v = moments_for(numels, seed + 2, spread)
    pools = {"p": Pool(numels, pdtype, packed, p), "g": Pool(numels, gdtype, packed, g)}
    if copy:
        pools["c"] = Pool(numels, torch.bfloat16, packed)
    full, states = states_of(numels)
    zs.moments_q8_encode(zs.Q8Moments(states, [from_np(x) for x in m], [from_np(x) for x in v]), seed=4)
    lst = zs.AdamWQ8Tensors(pools["p"].views, pools["g"].views, states, pools["c"].views if copy else None)
    key = ref.key_of(4, 0)
    m = [ref.stored(x, "m", k, key) for k, x in enumerate(m)]
    v = [ref.stored(x, "v", k, key) for k, x in enumerate(v)]
    return pools, full, states, lst, p, g, m, v


def check_step(numels, pools, states, p, g, m, v, hp, seed, coef):
    """One step's results against the definition; the new state in numpy."""
    s = zs.adamw_scalars(hp)
    key = ref.key_of(seed, hp.step)
    gm, gv = decoded(states, numels)
    bf16 = pools["p"].buffer.dtype == torch.bfloat16
    for k in range(len(numels)):
        m[k], v[k] = ref.new_moments(g[k], m[k], v[k], s, coef)
        want, u = ref.update64(p[k], m[k], v[k], s)
        # u: root, quotient, sum, reciprocal or quotient, products: at most 8 roundings or units of 2^-23; the
        # parameter: its product and its difference, 2^-24 of p and of the result
        bound = 16 * E24 * np.abs(u) + E24 * np.abs(p[k]) + E24 * (np.abs(p[k]) + np.abs(u))
        if bf16:
            bound = bound + 2.0 ** -8 * np.abs(want)
        got = pools["p"].views[k].cpu().double().numpy()
        assert (np.abs(got - want) <= bound).all(), k
        p[k] = pools["p"].views[k].cpu().float().numpy()
        if "c" in pools:
            assert same_bits(pools["c"].views[k], pools["p"].views[k].to(torch.bfloat16)), k
        m[k], v[k] = ref.stored(m[k], "m", k, key), ref.stored(v[k], "v", k, key)
        assert equal_values(gm[k], m[k]), (k, "exp_avg")
        assert equal_values(gv[k], v[k]), (k, "exp_avg_sq")


@pytest.mark.parametrize("pdtype,copy", [(torch.float32, False), (torch.float32, True), (torch.bfloat16, False)])
@pytest.mark.parametrize("gdtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("packed", [None, 0, 1])
@pytest.mark.parametrize("name", LISTS)
def test_step(name, packed, gdtype, pdtype, copy):
    print(name, packed, gdtype, pdtype, copy, flush=True)
    numels = LISTS[name]
    pools, full, states, lst, p, g, m, v = make(numels, pdtype, gdtype, copy, packed)
    norm = torch.tensor([6.25], dtype=torch.float64, device="cuda")
    for t, clip, seed in ((1, 0.0, 0), (2, 1.0, 5), (1000, 100.0, 0xFFFFFFFF)):
        hp = zs.AdamWConfig(**HP, max_norm=clip, step=t)
        zs.adamw_step_tensors_q8(hp, lst, seed=seed, norm_sq=norm if clip else None)
        coef = min(1.0, clip / (2.5 + 1e-6)) if clip else 1.0
        check_step(numels, pools, states, p, g, m, v, hp, seed, coef)
    assert guards_stand(full) and all(pool.guards_stand() for pool in pools.values())


def test_step_over_many_magnitudes():
    """Moments over 2^-40 of their block's largest, zero gradients, eps small
    and large, second moments that fall below the least code."""
    numels = [3000, 513]
    for eps in (1e-8, 1e-30, 1.0):
        pools, full, states, lst, p, g, m, v = make(numels, torch.float32, torch.float32, False, None, 71, 40.0)
        pools["g"].views[0][1000:2000] = 0
        g[0][1000:2000] = 0
        for t in (1, 2, 3):
            hp = zs.AdamWConfig(**{**HP, "eps": eps}, step=t)
            zs.adamw_step_tensors_q8(hp, lst, seed=t)
            check_step(numels, pools, states, p, g, m, v, hp, t, 1.0)


@pytest.mark.parametrize("pdtype", [torch.float32, torch.bfloat16])
def test_tiny_and_huge_gradients(pdtype):
    numels = [2048]
    for std in (1e-22, 1e-19, 1e-12, 1e4, 1e15):
        pools, full, states, lst, p, g, m, v = make(numels, pdtype, torch.float32, False, None)
        states[0].zero_()
        m[0][:], v[0][:] = 0, 0
        g[0] = (draws(numels, 3, 1.0)[0] * np.float32(std)).astype(np.float32)
        pools["g"].views[0].copy_(from_np(g[0]))
        for t in (1, 2):
            hp = zs.AdamWConfig(lr=1e-3, eps=1e-10, step=t)
            zs.adamw_step_tensors_q8(hp, lst)
            check_step(numels, pools, states, p, g, m, v, hp, 0, 1.0)


@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_non_finite(bad):
    """A non-finite norm leaves everything; without a norm a non-finite
    gradient makes its own block NaN and no other."""
    numels = [1000, 300]
    pools, full, states, lst, p, g, m, v = make(numels, torch.float32, torch.bfloat16, True, 1)
    before = [x.clone() for x in full] + [pool.buffer.clone() for pool in pools.values()]
    zs.adamw_step_tensors_q8(zs.AdamWConfig(**HP, max_norm=1.0), lst,
                             norm_sq=torch.tensor([bad], dtype=torch.float64, device="cuda"))
    after = full + [pool.buffer for pool in pools.values()]
    assert all(same_bits(a, b) for a, b in zip(before, after))
    pools["g"].views[0][300] = bad
    zs.adamw_step_tensors_q8(zs.AdamWConfig(**HP), lst)
    gm, gv = decoded(states, numels)
    nan = torch.isnan(gm[0]).cpu().numpy()
    assert nan[256:512].all() and not nan[:256].any() and not nan[512:].any() and not torch.isnan(gm[1]).any()
    assert np.array_equal(torch.isnan(gv[0]).cpu().numpy(), nan)
    par = torch.isnan(pools["p"].views[0]).cpu().numpy()
    assert par[300] and par.sum() == 1
    pools["g"].views[0][300] = 0
    zs.adamw_step_tensors_q8(zs.AdamWConfig(**HP, step=2), lst)        # the block stays NaN, its parameters follow
    par = torch.isnan(pools["p"].views[0]).cpu().numpy()
    assert par[256:512].all() and par.sum() == 256
    assert guards_stand(full)


def test_the_same_call_gives_the_same_bits_and_the_seed_matters():
    numels = [5000, 77]
    outs = []
    for seed in (1, 1, 2):
        pools, full, states, lst, *_ = make(numels, torch.float32, torch.bfloat16, True, None)
        for t in (1, 2, 3):
            zs.adamw_step_tensors_q8(zs.AdamWConfig(**HP, step=t), lst, seed=seed)
        gm, gv = decoded(states, numels)
        outs.append([x.clone() for x in gm + gv + pools["p"].views])
    assert all(same_bits(a, b) for a, b in zip(outs[0], outs[1]))
    assert not all(same_bits(a, b) for a, b in zip(outs[0], outs[2]))


def test_dev_scalars_and_a_captured_graph():
    numels = LISTS["many"] + [30_001]
    a = make(numels, torch.float32, torch.bfloat16, True, 1)
    b = make(numels, torch.float32, torch.bfloat16, True, 1)
    (pools, full, states, lst), (twin, tfull, tstates, eager) = a[:4], b[:4]
    norm = torch.zeros(1, dtype=torch.float64, device="cuda")
    grads = zs.GradTensors(pools["g"].views)
    ws = torch.empty(zs.grad_norm_sq_tensors_workspace_bytes(grads), dtype=torch.uint8, device="cuda")
    sc = torch.zeros(64, dtype=torch.uint8, device="cuda")

    def body():
        zs.grad_norm_sq_tensors(grads, 1 / 64, norm, ws)
        zs.adamw_step_tensors_q8_dev(sc, lst, norm_sq=norm)

    def scalars(t):
        hp = zs.AdamWConfig(**HP, max_norm=0.5, step=t)
        sc.copy_(torch.frombuffer(bytearray(zs.q8_scalars_bytes(hp, 17)), dtype=torch.uint8))
        return hp
    saved = [x.clone() for x in full], [pool.buffer.clone() for pool in pools.values()]
    scalars(1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        body()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for x, y in zip(full, saved[0]):
        x.copy_(y)
    for pool, y in zip(pools.values(), saved[1]):
        pool.buffer.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        body()
    for t in range(1, 5):
        for k, x in enumerate(draws(numels, 80 + t, 0.05 * t, True)):
            pools["g"].views[k].copy_(from_np(x))
            twin["g"].views[k].copy_(from_np(x))
        hp = scalars(t)
        graph.replay()
        enorm = torch.zeros(1, dtype=torch.float64, device="cuda")
        zs.grad_norm_sq_tensors(twin["g"].views, 1 / 64, enorm)
        zs.adamw_step_tensors_q8(hp, eager, seed=17, norm_sq=enorm)
        torch.cuda.synchronize()
        assert norm.item() == enorm.item()
        for k in ("p", "c"):
            assert same_bits(pools[k].buffer, twin[k].buffer), (t, k)
        for x, y in zip(decoded(states, numels), decoded(tstates, numels)):
            assert all(same_bits(i, j) for i, j in zip(x, y)), t


def test_a_tensor_past_2_31_elements():
    """Blocks on both sides of 2^31 and the last ones, their dither's index
    among what is checked (2^29 groups and more)."""
    n = (1 << 31) + 1025
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    state = torch.zeros(zs.moments_q8_bytes(n), dtype=torch.uint8, device="cuda")
    spans = [(0, 512), ((1 << 31) - 512, (1 << 31) + 512), (n - 513, n)]
    rng = np.random.default_rng(5)
    rows = []
    for lo, hi in spans:
        x = rng.standard_normal(hi - lo).astype(np.float32)
        g[lo:hi] = from_np(x).to(torch.bfloat16)
        rows.append(g[lo:hi].float().cpu().numpy())
    g[spans[1][0]:spans[1][1]] = from_np(rows[1]).to(torch.bfloat16)
    rows = [g[lo:hi].float().cpu().numpy() for lo, hi in spans]
    hp = zs.AdamWConfig(lr=1e-2, step=1)
    zs.adamw_step_tensors_q8(hp, zs.AdamWQ8Tensors([p], [g], [state]), seed=6)
    v = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    zs.moments_q8_decode(zs.Q8Moments([state], [m], [v]))
    s, key = zs.adamw_scalars(hp), ref.key_of(6, 1)
    for (lo, hi), x in zip(spans, rows):
        start = lo // 256 * 256                                # whole blocks
        gg = g[start:hi].float().cpu().numpy()
        zero = np.zeros(hi - start, np.float32)
        nm, nv = ref.new_moments(gg, zero, zero, s, 1.0)
        word = ref.words(hi - start, 0, key, first=start)
        assert equal_values(m[start:hi], ref.decode(*ref.encode(nm, "m", word), "m")), lo
        assert equal_values(v[start:hi], ref.decode(*ref.encode(nv, "v", word), "v")), lo
    assert int(torch.count_nonzero(v)) == sum(int((x != 0).sum()) for x in rows[:2]) + int(np.count_nonzero(rows[2]))


@pytest.mark.parametrize("pdtype", [torch.float32, torch.bfloat16])
def test_long_lists_off_cache_lines(pdtype):
    """More gradients than the last-level cache holds, as one tensor at odd
    offsets: stored, stepped and read out as the same tensor on 512-byte
    boundaries."""
    n = 130_000_003
    gen = torch.Generator(device="cuda").manual_seed(4)
    p, m, v, g = (torch.randn(n, generator=gen, device="cuda") * s for s in (0.05, 1e-3, 1e-3, 0.1))
    p, v, g = p.to(pdtype), v * v, g.bfloat16()
    done = []
    for off in (0, 1):
        ps, gs, ms, vs = (at_offset(x, off) for x in (p, g, m, v))
        state = torch.zeros(zs.moments_q8_bytes(n), dtype=torch.uint8, device="cuda")
        zs.moments_q8_encode(zs.Q8Moments([state], [ms], [vs]), seed=6)
        zs.adamw_step_tensors_q8(zs.AdamWConfig(**HP, step=4), zs.AdamWQ8Tensors([ps], [gs], [state]), seed=2)
        zs.moments_q8_decode(zs.Q8Moments([state], [ms], [vs]))
        done.append((state, ps, ms, vs))
    for a, b in zip(*done):
        assert torch.equal(a, b)


@pytest.mark.parametrize("numels", [
    [0] * 149 + [5, 600, 0, 7], [0] * 150 + [5, 600, 0, 7], [0] * 151 + [5], [3] + [0] * 400 + [513, 0, 0], [1] * 149 + [0, 0, 2],
    [1] * 150 + [0, 300], [512] * 300, [0] * 320, [700, 0] * 160], ids=lambda n: f"{len(n)}-{sum(n)}")
def test_empty_tensors_around_a_table(numels):
    """Tensors without elements take a place in the list (the dither knows it),
    also where a table ends; a step on them and a read-out of every second."""
    pools, full, states, lst, p, g, m, v = make(numels, torch.float32, torch.bfloat16, True, 1, seed=61)
    hp = zs.AdamWConfig(**HP, step=3)
    zs.adamw_step_tensors_q8(hp, lst, seed=9)
    check_step(numels, pools, states, p, g, m, v, hp, 9, np.float32(1.0))
    assert guards_stand(full) and all(pool.guards_stand() for pool in pools.values())
    out = Pool(numels, torch.float32, 1)
    zs.moments_q8_decode(zs.Q8Moments(states, [x if k % 2 else None for k, x in enumerate(out.views)], None, numels))
    assert out.guards_stand()
    for k, x in enumerate(out.views):
        if k % 2:
            assert equal_values(x, m[k]), k
        else:
            assert bool((x == 7.75).all()), k


@pytest.mark.parametrize("beta2", [0.95, 0.999, 0.999999])
@pytest.mark.parametrize("eps", [2.0 ** -41, 2.0 ** -40, 1e-12, 2.0 ** -38, 2.0 ** -36, 2.0 ** -34, 2.0 ** -32, 2.0 ** -30, 1e-8])
def test_the_update_s_bound_at_small_second_moments(eps, beta2):
    """From a zero parameter, whose step is then all of it: second moments on
    both sides of the least normal number, eps around where the form changes."""
    print(eps, beta2, flush=True)
    n = 4096
    v = np.geomspace(2.0 ** -140, 2.0 ** -100, n)
    sign = np.where(np.arange(n) % 3 == 0, -1.0, 1.0)
    check_update_from_zero(sign * np.sqrt(v / (1 - beta2)), eps, beta2, lr=1e-3)


@pytest.mark.parametrize("eps", [1.0, 2.0 ** 99, 2.0 ** 100, 2.0 ** 101, 2.0 ** 125, 2.0 ** 126, 2.0 ** 127, 3.4e38])
def test_the_update_s_bound_at_large_eps(eps):
    """eps up to the largest number, whose reciprocal is subnormal."""
    print(eps, flush=True)
    check_update_from_zero(np.geomspace(1e10, 1e18, 2048), eps, 0.999, lr=1e12)


def check_update_from_zero(gradients, eps, beta2, lr):
    """Steps 1 and 1000 from zero moments and parameters: the header's 8 * 2^-24
    of the quotient, and half a step of the product with step_size, 2^-24."""
    g = gradients.astype(np.float32)
    n = g.size
    zero = np.zeros(n, np.float32)
    for step in (1, 1000):
        hp = zs.AdamWConfig(lr=lr, beta1=0.9, beta2=beta2, eps=eps, step=step)
        p = torch.zeros(n, device="cuda")
        state = torch.zeros(zs.moments_q8_bytes(n), dtype=torch.uint8, device="cuda")
        zs.adamw_step_tensors_q8(hp, zs.AdamWQ8Tensors([p], [from_np(g)], [state]))
        s = zs.adamw_scalars(hp)
        m, v = ref.new_moments(g, zero, zero, s, 1.0)
        _, u = ref.update64(zero, m, v, s)
        assert (np.abs(u) > 2.0 ** -100).all()
        off = np.abs(p.cpu().double().numpy() + u) / np.abs(u) / E24
        assert off.max() <= 8 + 1 + 2.0 ** -19, (step, off.max())     # their product's term of second order
