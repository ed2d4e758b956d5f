"""Operators over a model's matrices and its whole gradient, as cases to time and compare: norms and clipping of lists of
mixed precision, products with a scaled residual (general and symmetric), orthogonalisation by Newton-Schulz steps and the
momentum update that uses it.

A case is a decoder's projection matrices (some depth and width) and what the operator does with them.  Matrices of one
shape lie one behind the other, the shapes one behind the other in a buffer per kind: every stack on a 256-element
boundary, or ("packed") everything back to back from an odd offset on.  Clipping takes a model's whole list, vectors and
embedding among it, matrices in bf16 beside vectors in fp32.
"""
import math

import torch

own = False

LR, MOMENTUM, DECAY, SCALE, MAX_NORM, EPS = 3e-4, 0.95, 0.1, 1.0 / 64, 1.0, 1e-7
CLIP_NORM = 0.01                                 # of the clipping cases: most of their norms are above it
A, B, C, STEPS = 3.4445, -4.7750, 2.0315, 5      # the quintic and how often it is applied
ALPHA, BETA = 0.05, 0.95                         # a preconditioner's running statistics
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def case_of(name, op, layers, hidden, ffn, kv, vocab=0, odd=0, grad="bf16", param="f32", out="f32", copy=False, clip=False,
            packed=False, nesterov=True):
    return {"name": name, "op": op, "layers": layers, "hidden": hidden, "ffn": ffn, "kv": kv, "vocab": vocab, "odd": odd,
            "grad": grad, "param": param, "out": out, "copy": copy, "clip": clip, "packed": packed, "nesterov": nesterov}


def listed():
    return [
        # one small decoder layer, its embedding and an odd projection: latency
        case_of("clip small", "clip", 1, 256, 600, 256, 1000, 103 * 197, out="bf16"),
        # 7B's depth at a sixteenth of its width, odd sizes back to back
        case_of("clip deep packed", "clip", 32, 251, 683, 251, 1000, out="bf16", packed=True),
        # four layers of a 7B-style model: bf16 gradients out as unscaled fp32 ones for a step that wants these
        case_of("clip 7B layers", "clip", 4, 4096, 11008, 4096),
        # a preconditioner's statistics L = 0.95 L + 0.05 G G^T on the short side: many small odd matrices, one 7B layer
        case_of("gram deep packed", "gram", 32, 251, 683, 251, packed=True),
        case_of("gram 7B layer", "gram", 1, 4096, 11008, 4096),
        # a preconditioner applied to the gradients with their residual, P G + G
        case_of("product small", "product", 1, 256, 600, 64, out="bf16"),
        case_of("product 7B layer", "product", 1, 4096, 11008, 4096, out="bf16"),
        # orthogonal factors of a list of matrices
        case_of("orthogonalize small", "orthogonalize", 1, 256, 600, 64, grad="f32"),
        case_of("orthogonalize 13B layer", "orthogonalize", 1, 5120, 13824, 5120),
        # the whole momentum step: a small model, 224 odd matrices with bf16 parameters, two 7B layers with fp32 masters
        case_of("muon small", "muon", 1, 256, 600, 256, grad="f32"),
        case_of("muon deep packed", "muon", 32, 251, 683, 251, param="bf16", packed=True, nesterov=False),
        case_of("muon 7B layers", "muon", 2, 4096, 11008, 4096, copy=True, clip=True),
    ]


def stacks(case):
    """(count, rows, cols) of each shape of projection matrix: q and o; k and v; gate and up; down."""
    n, h, f, kv = case["layers"], case["hidden"], case["ffn"], case["kv"]
    square = [(4 * n, h, h)] if kv == h else [(2 * n, h, h), (2 * n, kv, h)]
    return square + [(2 * n, f, h), (n, h, f)]


def vectors(case):
    """Elements of the fp32 tensors beside the matrices (clipping): norm vectors, the embedding, an odd one."""
    return [case["hidden"]] * (2 * case["layers"] + 1) + [n for n in (case["vocab"] * case["hidden"], case["odd"]) if n]


def flops_of(case):
    op, total = case["op"], 0
    for count, rows, cols in stacks(case):
        m, n = min(rows, cols), max(rows, cols)
        if op == "gram":
            total += count * m * m * n
        elif op == "product":
            total += count * 2 * rows * rows * cols
        elif op in ("orthogonalize", "muon"):
            total += count * STEPS * (3 * m * m * n + m * m * m)
        else:
            total += count * 5 * m * n
    return total


def draw(rng):
    """Models of 1e4 to 4e8 parameters for clipping, fewer where the products of wide matrices cost more than the largest
    listed case; the width goes by the size, odd widths among them."""
    op = rng.choice(["clip", "gram", "product", "orthogonalize", "muon", "muon"])
    most = max(flops_of(c) for c in listed() if c["op"] == op)
    while True:
        target = math.exp(rng.uniform(math.log(1e4), math.log(4e8)))
        layers = max(1, round(math.exp(rng.uniform(0.0, math.log(32)))))
        h = max(5, int(math.sqrt(target / (12 * layers))))
        h = h if rng.random() < 0.4 else max(8, h // 64 * 64 if h >= 64 else h // 8 * 8)
        f = max(7, int(h * rng.uniform(2.5, 3.6)))
        kv = max(1, h // rng.choice([1, 1, 4, 8]))
        param = rng.choice(["f32", "f32", "bf16"])
        case = case_of("", op, layers, h, f, kv, rng.choice([0, rng.randrange(7, 1000)]) if op == "clip" else 0,
                       rng.choice([0, 1, rng.randrange(2, 70000)]) if op == "clip" else 0, grad=rng.choice(["bf16", "f32"]),
                       param=param, out=rng.choice(["bf16", "f32"]), copy=param == "f32" and rng.random() < 0.6,
                       clip=rng.random() < 0.5, packed=rng.random() < 0.4, nesterov=rng.random() < 0.7)
        if flops_of(case) <= most:
            return {k: v for k, v in case.items() if k != "name"}


def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    g, o, flops = size[case["grad"]], size[case["out"]], flops_of(case)
    n = sum(count * rows * cols for count, rows, cols in stacks(case))
    if op == "clip":
        extra = sum(vectors(case))
        return {"bytes": n * (g + o) + extra * (4 + size[case["out"]]), "flops": flops}
    if op == "gram":
        square = sum(count * min(rows, cols) ** 2 for count, rows, cols in stacks(case))
        return {"bytes": n * g + square * 8, "flops": flops}
    if op == "product":
        square = sum(count * rows * rows for count, rows, cols in stacks(case))
        return {"bytes": square * g + n * (g + o), "flops": flops}
    if op == "orthogonalize":
        return {"bytes": n * (g + 2), "flops": flops}
    return {"bytes": n * (g + 8 + 2 * size[case["param"]] + (2 if case["copy"] else 0)), "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def layout(case, shapes):
    """The offset of each stack in a buffer that holds (count, rows, cols) of every shape, and the buffer's length."""
    at, out = (1 if case["packed"] else 0), []
    for count, rows, cols in shapes:
        out.append(at)
        at += count * rows * cols
        at = at if case["packed"] else -(-at // 256) * 256
    return out, at


def views(case, buffer, shapes):
    at, _ = layout(case, shapes)
    return [buffer[a:a + n * r * c].view(n, r, c) for a, (n, r, c) in zip(at, shapes)]


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    shapes, op = stacks(case), case["op"]
    s = {"case": case, "shapes": shapes}

    def normal(std, *shape):
        return torch.empty(*shape, device=dev).normal_(0.0, std, generator=gen)

    def buffer(dtype, shapes=shapes):
        return torch.zeros(layout(case, shapes)[1], dtype=dtype, device=dev)

    def gradients(std, dtype):
        """A few strong directions over noise, as sums of outer products over a batch of tokens are."""
        x = buffer(torch.float32)
        for v, (n, r, c) in zip(views(case, x, shapes), shapes):
            k = min(16, r, c)
            fade = 4.0 / torch.arange(1, k + 1, device=dev)
            v.copy_(torch.bmm(normal(std, n, r, k) * fade, normal(1.0, n, k, c)))
            v += normal(std, n, r, c)
        return x.to(dtype)

    s["grad"] = gradients(1e-3, DTYPES[case["grad"]])
    if op == "clip":
        at, s["vectors"] = 0, vectors(case)
        s["grad_vectors"] = normal(1e-3, sum(s["vectors"]))
        s["out"], s["out_vectors"] = buffer(DTYPES[case["out"]]), torch.zeros(sum(s["vectors"]), dtype=DTYPES[case["out"]],
                                                                               device=dev)
        s["total"] = torch.zeros(1, dtype=torch.float64, device=dev)
    elif op == "gram":
        s["squares"] = [(n, min(r, c), min(r, c)) for n, r, c in shapes]
        s["stat"] = buffer(torch.float32, s["squares"])
        for v in views(case, s["stat"], s["squares"]):
            x = normal(1e-3, v.shape[0], v.shape[1], 24)
            v.copy_(torch.bmm(x, x.transpose(1, 2).contiguous()))
    elif op == "product":
        s["squares"] = [(n, r, r) for n, r, c in shapes]
        s["pre"] = normal(0.02, layout(case, s["squares"])[1]).to(DTYPES[case["grad"]])
        s["out"] = buffer(DTYPES[case["out"]])
    elif op == "orthogonalize":
        s["out"] = buffer(torch.bfloat16)
    else:
        s["param"] = normal(0.02, s["grad"].numel()).to(DTYPES[case["param"]])
        s["copy"] = s["param"].to(torch.bfloat16) if case["copy"] else None
        s["momentum"] = gradients(5e-4 * SCALE, torch.float32)
        s["norm"] = (s["grad"].float() * SCALE).double().square().sum().reshape(1)
    if own:
        handles(s)
    return s


def matrices(s, buffer, shapes=None):
    """Every matrix of a buffer, in order."""
    return None if buffer is None else [m for v in views(s["case"], buffer, shapes or s["shapes"]) for m in v]


def handles(s):
    """The lists that a program marshals once, and its workspaces."""
    import fsdp_sharded_optimizer_amd as zs
    op, dev = s["case"]["op"], "cuda"
    if op == "clip":
        tensors = matrices(s, s["grad"]) + list(s["grad_vectors"].split(s["vectors"]))
        outs = matrices(s, s["out"]) + list(s["out_vectors"].split(s["vectors"]))
        s["list"], s["to"] = zs.MixedTensors(tensors), zs.MixedTensors(outs)
        s["norms"] = torch.zeros(len(tensors), dtype=torch.float64, device=dev)
        need = zs.grad_norms_sq_tensors_workspace_bytes(s["list"])
    elif op == "gram":
        s["list"] = zs.GramMatrices(matrices(s, s["grad"]), matrices(s, s["stat"], s["squares"]),
                                    matrices(s, s["stat"], s["squares"]))
        need = zs.gram_add_matrices_workspace_bytes(s["list"])
    elif op == "product":
        s["list"] = zs.ProductMatrices(matrices(s, s["pre"], s["squares"]), matrices(s, s["grad"]), matrices(s, s["out"]),
                                       matrices(s, s["grad"]))
        need = zs.product_add_matrices_workspace_bytes(s["list"])
    elif op == "orthogonalize":
        s["list"] = zs.OrthogonalizeMatrices(matrices(s, s["grad"]), matrices(s, s["out"]))
        need = zs.orthogonalize_matrices_workspace_bytes(s["list"])
    else:
        s["list"] = zs.MuonMatrices(matrices(s, s["param"]), matrices(s, s["grad"]), matrices(s, s["momentum"]),
                                    matrices(s, s["copy"]), scale="rms")
        need = zs.muon_step_matrices_workspace_bytes(s["list"])
    s["workspace"] = torch.empty(max(8, need), dtype=torch.uint8, device=dev)


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def transposed(x):
    return x.transpose(1, 2).contiguous()


def short_gram(x):
    """X X^T or X^T X of every matrix of a stack, whichever is smaller."""
    x = x if x.shape[1] <= x.shape[2] else transposed(x)
    return torch.bmm(x, transposed(x))


def plain_clip(s):
    shapes, g = s["shapes"], s["grad"].float() * SCALE
    v = s["grad_vectors"] * SCALE
    each = [x.double().square().sum((1, 2)) for x in views(s["case"], g, shapes)]
    each += [x.double().square().sum().reshape(1) for x in v.split(s["vectors"])]
    norms = torch.cat(each)
    total = norms.sum().reshape(1)
    coef = (CLIP_NORM / (total.sqrt() + 1e-6)).clamp(max=1.0).float()
    s["out"].copy_(g * coef)
    s["out_vectors"].copy_(v * coef)
    return {"norms": norms, "total": total, "out": s["out"], "vectors": s["out_vectors"]}


def plain_orthogonal(x):
    """The orthogonal factor, nearly, of every matrix of a stack."""
    tall = x.shape[1] > x.shape[2]
    x = transposed(x) if tall else x
    x = x / torch.linalg.vector_norm(x.double(), dim=(1, 2), keepdim=True).clamp(min=EPS).float()
    for _ in range(STEPS):
        gram = torch.bmm(x, transposed(x))
        x = A * x + torch.bmm(B * gram + C * torch.bmm(gram, gram), x)
    return transposed(x) if tall else x


def plain_muon(s):
    case = s["case"]
    g = s["grad"].float() * SCALE
    if case["clip"]:
        g = g * (MAX_NORM / (s["norm"].sqrt() + 1e-6)).clamp(max=1.0).float()
    m = s["momentum"].mul_(MOMENTUM).add_(g * (1 - MOMENTUM))
    u = m * MOMENTUM + g * (1 - MOMENTUM) if case["nesterov"] else m
    for x, p in zip(views(case, u, s["shapes"]), views(case, s["param"], s["shapes"])):
        step = LR * 0.2 * math.sqrt(max(x.shape[1:]))
        p.copy_(p.float() * (1 - LR * DECAY) - plain_orthogonal(x) * step)
    if s["copy"] is not None:
        s["copy"].copy_(s["param"])


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return run_own(s, op)
    if op == "clip":
        return plain_clip(s)
    if op == "gram":
        for x, stat in zip(views(s["case"], s["grad"], s["shapes"]), views(s["case"], s["stat"], s["squares"])):
            stat.copy_(BETA * stat + ALPHA * short_gram(x.float()))
        return s["stat"]
    if op == "product":
        for x, p, y in zip(views(s["case"], s["grad"], s["shapes"]), views(s["case"], s["pre"], s["squares"]),
                           views(s["case"], s["out"], s["shapes"])):
            y.copy_(torch.bmm(p.float(), x.float()) + x.float())
        return s["out"]
    if op == "orthogonalize":
        for x, y in zip(views(s["case"], s["grad"], s["shapes"]), views(s["case"], s["out"], s["shapes"])):
            y.copy_(plain_orthogonal(x.float()))
        return s["out"]
    plain_muon(s)
    return {"param": s["param"], "copy": s["copy"], "momentum": s["momentum"]}


def run_own(s, op):
    import fsdp_sharded_optimizer_amd as zs
    ws = s["workspace"]
    if op == "clip":
        zs.grad_norms_sq_tensors(s["list"], SCALE, s["total"], norms=s["norms"], workspace=ws)
        zs.grad_clip_tensors(s["list"], s["to"], SCALE, CLIP_NORM, s["total"])
        return {"norms": s["norms"], "total": s["total"], "out": s["out"], "vectors": s["out_vectors"]}
    if op == "gram":
        zs.gram_add_matrices(s["list"], alpha=ALPHA, beta=BETA, workspace=ws)
        return s["stat"]
    if op == "product":
        zs.product_add_matrices(s["list"], alpha=1.0, beta=1.0, workspace=ws)
        return s["out"]
    if op == "orthogonalize":
        zs.orthogonalize_matrices(s["list"], steps=STEPS, coefficients=(A, B, C), eps=EPS, workspace=ws)
        return s["out"]
    hp = zs.MuonConfig(lr=LR, momentum=MOMENTUM, nesterov=s["case"]["nesterov"], weight_decay=DECAY, ns_steps=STEPS,
                       coefficients=(A, B, C), eps=EPS, grad_scale=SCALE, max_norm=MAX_NORM)
    zs.muon_step_matrices(hp, s["list"], norm_sq=s["norm"] if s["case"]["clip"] else None, workspace=ws)
    return {"param": s["param"], "copy": s["copy"], "momentum": s["momentum"]}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact_orthogonal(u):
    """One matrix; the polynomial of its singular values by the other association, S X first and then S (S X)."""
    x = u / max(float(u.square().sum().sqrt()), EPS)
    for _ in range(STEPS):
        if u.shape[0] <= u.shape[1]:
            gram = x @ x.t().contiguous()
            once = gram @ x
            x = A * x + B * once + C * (gram @ once)
        else:
            gram = x.t().contiguous() @ x
            once = x @ gram
            x = A * x + B * once + C * (once @ gram)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op, g = case["op"], s["grad"].double()
    if op == "clip":
        out, norms = g * SCALE, []
        v = s["grad_vectors"].double() * SCALE
        for x in matrices(s, out) + list(v.split(s["vectors"])):
            norms.append(torch.linalg.vector_norm(x).square())
        total = sum(norms)
        coef = min(1.0, CLIP_NORM / (math.sqrt(float(total)) + 1e-6))
        return {"norms": torch.stack(norms), "total": total.reshape(1), "out": out * coef, "vectors": v * coef}
    if op == "gram":
        stat = s["stat"].double()
        for x, y in zip(matrices(s, g), matrices(s, stat, s["squares"])):
            x = x if x.shape[0] <= x.shape[1] else x.t().contiguous()
            y.mul_(BETA).add_(x @ x.t().contiguous(), alpha=ALPHA)
        return stat
    out = torch.zeros_like(g)
    if op == "product":
        for p, x, y in zip(matrices(s, s["pre"].double(), s["squares"]), matrices(s, g), matrices(s, out)):
            y.copy_(p @ x)
        return out.add_(g)
    if op == "orthogonalize":
        for x, y in zip(matrices(s, g), matrices(s, out)):
            y.copy_(exact_orthogonal(x))
        return out
    g *= SCALE
    if case["clip"]:
        g *= min(1.0, MAX_NORM / (float(g.square().sum().sqrt()) + 1e-6))
    momentum = MOMENTUM * s["momentum"].double() + (1 - MOMENTUM) * g
    param = s["param"].double()
    u = MOMENTUM * momentum + (1 - MOMENTUM) * g if case["nesterov"] else momentum
    for x, p in zip(matrices(s, u), matrices(s, param)):
        p.mul_(1 - LR * DECAY).sub_(exact_orthogonal(x), alpha=LR * 0.2 * math.sqrt(max(x.shape)))
    return {"param": param, "copy": param.clone() if case["copy"] else None, "momentum": momentum}
