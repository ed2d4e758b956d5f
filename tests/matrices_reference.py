"""Plain forms, in 64 bits, of the calls over lists of matrices, and their error bounds."""
import torch

COEFFICIENTS = (3.4445, -4.7750, 2.0315)

# Error of a result of orthogonalize_matrices before its last rounding, relative in the
# Frobenius norm.  One rounding to fp16 is off by 2^-11 at most, by 2^-11 / sqrt(3) * 0.7 =
# 2e-4 rms.  A step rounds X (which enters S twice), S and P = b S + c S^2; at singular
# values near 1 they weigh 2 (|b| + 2 |c|) = 18, |b| + 2 |c| = 9 and |P| = 3, together 20 *
# 2e-4 = 4e-3 of what a rounding of every singular direction alike would do; the next step
# multiplies it by |f'(1)| = 0.7.  Small singular values come through a X, which is not rounded.
# Short sides up to 64, with too few singular values for roundings to average, are formed from
# S and a product of polynomials in fp32, with X and that as pairs of 22 bits: S is off by about
# 2^-23, and the product moves by up to a^5 (|b| / a) (1 + a^2 + ... + a^8) = 1.5e7 times that near
# s = 0: 1.8 sigma for sigma < 1e-3, and 1e-5 where all singular values count.
NS_BOUND = 4e-3
BF16 = 2.0 ** -8          # half a step of bf16, relative
FP32 = 2.0 ** -24


def orthogonal(x, steps=5, coefficients=COEFFICIENTS, eps=1e-7):
    """X <- a X + (b S + c S^2) X of one matrix, `steps` times."""
    a, b, c = coefficients
    x = x.double()
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    x = x / max(float(x.square().sum().sqrt()), eps)
    for _ in range(steps):
        s = x @ x.t().contiguous()
        x = a * x + (b * s + c * (s @ s)) @ x
    return x.t().contiguous() if tall else x


def momentum(m, g, mu, nesterov, scale=1.0, coef=1.0):
    """The new momentum and u, with the roundings of the kernel (fp32, one per operation)."""
    f = lambda v: torch.tensor(v, dtype=torch.float32, device=m.device)  # noqa: E731
    g = g.float() * f(scale) * f(coef)
    new = f(mu) * m + f(1 - mu) * g
    return new, (f(mu) * new + f(1 - mu) * g if nesterov else new)


def product_bound(a, b, k, alpha, beta, c, split):
    """Elementwise bound of alpha a b + beta c formed in fp32: sums of k products, and
    the three roundings after them; split: fp32 inputs as two bf16 values each."""
    size = a.double().abs() @ b.double().abs() * abs(alpha)
    rest = (c.double().abs() * abs(beta)) if c is not None else 0.0
    return (k * (3 if split else 1) + 4) * FP32 * size + 4 * FP32 * rest + (3 * 2.0 ** -16 * size if split else 0.0)


def matrix(rows, cols, seed, kind="noise", dtype=torch.float32, device="cuda"):
    """A matrix as gradients are: noise, a few directions over noise, of rank one, or fading."""
    gen = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device=device)  # noqa: E731
    if kind == "noise":
        x = r(rows, cols)
    elif kind == "directions":
        x = r(rows, 4) @ r(4, cols) + 1e-2 * r(rows, cols)
    elif kind == "rank one":
        x = r(rows, 1) @ r(1, cols)
    else:
        k = min(rows, cols)
        x = (torch.linalg.qr(r(rows, k))[0] / torch.arange(1, k + 1, device=device)) @ torch.linalg.qr(r(cols, k))[0].t().contiguous()
    return (x * 1e-3).to(dtype).contiguous()


def far(x, y):
    """Relative distance in the Frobenius norm."""
    y = y.double()
    return float((x.double() - y).norm() / y.norm()) if float(y.norm()) else float(x.double().norm())
