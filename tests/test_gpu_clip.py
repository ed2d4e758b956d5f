"""Norms and clipping over lists of mixed precision, against plain forms in 64 bits."""
import pytest
import torch

import fsdp_sharded_optimizer_amd as zs

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16
# around the tiles of the norm (4096 fp32, 8192 bf16) and of the clipping (4096), empty ones, odd ones
SIZES = [1, 0, 3, 4, 255, 4095, 4096, 4097, 8191, 8192, 8193, 0, 70001, 300000, 5]


def lists(sizes, seed=0, std=1e-2):
    """Views of two buffers, at odd offsets: (tensors, buffers)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    bufs = {dt: torch.randn(sum(sizes) + 7, generator=gen, device="cuda").mul_(std).to(dt) for dt in (F32, BF16)}
    at, out = {F32: 1, BF16: 3}, []
    for k, n in enumerate(sizes):
        dt = (F32, BF16)[(k * 7 // 3) % 2]
        out.append(bufs[dt][at[dt]:at[dt] + n])
        at[dt] += n
    return out, bufs


def norm_of(ts, scale):
    # squares of binary32 values are exact in binary64, so the sums alone round: 2^-53 a step
    return torch.stack([(t.float() * torch.tensor(scale, device="cuda")).double().square().sum() for t in ts])


@pytest.mark.parametrize("scale", [1.0, 1.0 / 64, 3.0])
def test_norms(scale):
    ts, _ = lists(SIZES)
    out = torch.full((1,), -1.0, dtype=torch.float64, device="cuda")
    norms = torch.full((len(ts) + 1,), -1.0, dtype=torch.float64, device="cuda")
    zs.grad_norms_sq_tensors(ts, scale, out, norms=norms[:-1])
    want = norm_of(ts, scale)
    # a sum of n terms of one sign in any order: n 2^-53 relative at most
    assert torch.allclose(norms[:-1], want, rtol=3e5 * 2.0 ** -53, atol=0) and norms[-1] == -1.0
    assert norms[1] == 0 and torch.allclose(out[0], want.sum(), rtol=5e5 * 2.0 ** -53, atol=0)
    again = torch.empty_like(out)
    zs.grad_norms_sq_tensors(zs.MixedTensors(ts), scale, again)      # without the norms: the same bits
    assert torch.equal(out, again)


def test_norms_of_lists_longer_than_a_table():
    sizes = [0 if k % 97 == 5 else 1 + k % 13 for k in range(2500)]
    ts, _ = lists(sizes)
    out, norms = torch.empty(1, dtype=torch.float64, device="cuda"), torch.empty(2500, dtype=torch.float64, device="cuda")
    zs.grad_norms_sq_tensors(ts, 0.5, out, norms=norms)
    want = norm_of(ts, 0.5)
    assert torch.allclose(norms, want, rtol=1e-14, atol=0) and torch.allclose(out[0], want.sum(), rtol=1e-12, atol=0)


def test_an_empty_list_and_lists_without_elements():
    for ts in ([], [torch.empty(0, device="cuda"), torch.empty(0, device="cuda", dtype=BF16)]):
        out = torch.full((1,), 7.0, dtype=torch.float64, device="cuda")
        norms = torch.full((2,), 7.0, dtype=torch.float64, device="cuda")
        zs.grad_norms_sq_tensors(ts, 1.0, out, norms=norms)
        assert out.item() == 0.0 and norms.tolist() == ([0.0, 0.0] if ts else [7.0, 7.0])
        zs.grad_clip_tensors(ts, max_norm=1.0, norm_sq=out)


def clipped(t, scale, coef, dtype):
    f = lambda v: torch.tensor(v, dtype=F32, device="cuda")  # noqa: E731
    return (t.float() * f(scale) * f(coef)).to(dtype)


@pytest.mark.parametrize("max_norm", [0.0, 0.5, 1e9])
@pytest.mark.parametrize("to", [F32, BF16, "mixed"])
def test_clip(max_norm, to):
    ts, src = lists(SIZES)
    kept = {dt: b.clone() for dt, b in src.items()}
    norm = torch.empty(1, dtype=torch.float64, device="cuda")
    zs.grad_norms_sq_tensors(ts, 1.0 / 3, norm)
    outs, bufs = lists(SIZES, seed=1)
    before = {dt: b.clone() for dt, b in bufs.items()}
    if to != "mixed":
        bufs = {to: torch.full((sum(SIZES) + 9,), 7.0, dtype=to, device="cuda")}
        before = {to: bufs[to].clone()}
        outs = list(bufs[to][5:-4].split(SIZES))
    zs.grad_clip_tensors(ts, outs, 1.0 / 3, max_norm, norm, extra_norm_sq=2.0)
    coef = float((max_norm / ((norm + 2.0).sqrt() + 1e-6)).clamp(max=1.0).float()) if max_norm else 1.0
    for t, y in zip(ts, outs):
        assert torch.equal(y, clipped(t, 1.0 / 3, coef, y.dtype))
    assert all(torch.equal(src[dt], kept[dt]) for dt in src)
    written = sum(SIZES) if to != "mixed" else None
    for dt, b in bufs.items():
        n = written if written is not None else sum(t.numel() for t in outs if t.dtype == dt)
        first = 5 if to != "mixed" else {F32: 1, BF16: 3}[dt]
        assert torch.equal(b[:first], before[dt][:first]) and torch.equal(b[first + n:], before[dt][first + n:])


@pytest.mark.parametrize("scale,max_norm", [(1.0, 0.25), (1.0, 0.0), (0.125, 0.25), (1.0, 1e9)])
def test_clip_in_place(scale, max_norm):
    ts, _ = lists(SIZES)
    norm = torch.empty(1, dtype=torch.float64, device="cuda")
    lst = zs.MixedTensors(ts)
    zs.grad_norms_sq_tensors(lst, scale, norm)
    coef = float((max_norm / (norm.sqrt() + 1e-6)).clamp(max=1.0).float()) if max_norm else 1.0
    want = [clipped(t, scale, coef, t.dtype) for t in ts]
    zs.grad_clip_tensors(lst, None, scale, max_norm, norm)
    assert all(torch.equal(a, b) for a, b in zip(ts, want))


def test_clip_on_a_non_finite_norm_changes_nothing():
    ts, bufs = lists(SIZES)
    ts[5][17] = float("inf")
    norm = torch.empty(1, dtype=torch.float64, device="cuda")
    before = {dt: b.clone() for dt, b in bufs.items()}
    zs.grad_norms_sq_tensors(ts, 1.0, norm)
    assert not torch.isfinite(norm).item()
    zs.grad_clip_tensors(ts, None, 0.5, 1.0, norm)
    assert all(torch.equal(bufs[dt], before[dt]) for dt in bufs)


def test_clip_scales_without_a_norm():
    ts, _ = lists(SIZES)
    want = [clipped(t, 0.5, 1.0, t.dtype) for t in ts]
    zs.grad_clip_tensors(ts, grad_scale=0.5, max_norm=1.0)
    assert all(torch.equal(a, b) for a, b in zip(ts, want))


def test_captured_norms_and_clip_replay():
    ts, bufs = lists(SIZES)
    outs = [torch.empty_like(t, dtype=F32) for t in ts]
    lst, to = zs.MixedTensors(ts), zs.MixedTensors(outs)
    norm = torch.empty(1, dtype=torch.float64, device="cuda")
    norms = torch.empty(len(ts), dtype=torch.float64, device="cuda")
    ws = torch.empty(zs.grad_norms_sq_tensors_workspace_bytes(lst), dtype=torch.uint8, device="cuda")

    def step():
        zs.grad_norms_sq_tensors(lst, 0.5, norm, norms=norms, workspace=ws)
        zs.grad_clip_tensors(lst, to, 0.5, 0.25, norm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        for b in bufs.values():
            b.mul_(1.5)
        graph.replay()
        got = [norm.clone(), norms.clone()] + [t.clone() for t in outs]
        torch.cuda.synchronize()
        step()
        assert all(torch.equal(a, b) for a, b in zip(got, [norm, norms] + outs)), k
