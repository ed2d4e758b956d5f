"""The operators over many tensors at once: the gradient norm, AdamW with fp32 or 8-bit moments, and the 8-bit moments'
conversions, as cases to time and compare.

A case is a model's list of tensors (a decoder of some depth and width, in module order) and what the operator does with
it.  The tensors are views of one buffer per kind, the way flat-parameter frameworks and bucketed allocators hold them:
each on a 256-element boundary, or ("packed") one behind the other from an odd offset on.  The buffers are the outputs.

8-bit moments are returned as the values they stand for, which bf16 holds exactly (4 significant bits).
"""
import math

import torch

own = False

LR, BETA1, BETA2, EPS, DECAY, SCALE, MAX_NORM = 3e-4, 0.9, 0.95, 1e-8, 0.1, 1.0 / 64, 1.0
BLOCK = 256          # elements that share a scale in the 8-bit moments
GOLDEN, MULT1, MULT2 = 0x9E3779B9, 0x6A09E667, 0xBB67AE85
MASK = 0xFFFFFFFF
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def case_of(name, op, layers, hidden, ffn, kv, vocab, odd, grad="bf16", param="f32", copy=False, clip=False, packed=False,
            moments="f32"):
    return {"name": name, "op": op, "layers": layers, "hidden": hidden, "ffn": ffn, "kv": kv, "vocab": vocab, "odd": odd,
            "grad": grad, "param": param, "copy": copy, "clip": clip, "packed": packed, "moments": moments}


def listed():
    return [
        # one small decoder layer, its embedding and an odd projection (1,000,003 parameters in 12 tensors): latency
        case_of("norm small", "norm", 1, 256, 600, 256, 1000, 103 * 197, grad="f32"),
        # one block of a 70B-style model (855M parameters in 9 tensors, two of them norm vectors)
        case_of("norm 70B block", "norm", 1, 8192, 28672, 1024, 0, 0),
        # the small model's step: launch bound
        case_of("adamw small", "step", 1, 256, 600, 256, 1000, 103 * 197, grad="f32"),
        # four layers of a 7B-style model: fp32 masters with their bf16 re-casts, clipped
        case_of("adamw 7B layers", "step", 4, 4096, 11008, 4096, 0, 0, copy=True, clip=True),
        # 7B's depth (290 tensors) at a sixteenth of its width, odd sizes back to back, bf16 parameters updated in place
        case_of("adamw deep packed", "step", 32, 251, 683, 251, 1000, 0, grad="f32", param="bf16", clip=True, packed=True),
        # two layers of a 13B-style model on fp32 gradients (accumulated over micro-batches)
        case_of("adamw 13B layers", "step", 2, 5120, 13824, 5120, 0, 0, grad="f32", copy=True),
        # the same four with both moments in 8 bits
        case_of("adamw q8 small", "step_q8", 1, 256, 600, 256, 1000, 103 * 197, grad="f32"),
        case_of("adamw q8 7B layers", "step_q8", 4, 4096, 11008, 4096, 0, 0, copy=True, clip=True),
        case_of("adamw q8 deep packed", "step_q8", 32, 251, 683, 251, 1000, 0, copy=True, clip=True, packed=True),
        case_of("adamw q8 70B block", "step_q8", 1, 8192, 28672, 1024, 0, 0, param="bf16"),
        # moments into 8 bits and back: a checkpoint's load and save
        case_of("moments q8 small", "codec", 1, 256, 600, 256, 1000, 103 * 197),
        case_of("moments q8 13B layer", "codec", 1, 5120, 13824, 5120, 0, 0, moments="bf16"),
    ]


def numels(case):
    """Elements of each tensor, in module order."""
    h, f, kv = case["hidden"], case["ffn"], case["kv"]
    layer = [h * h, kv * h, kv * h, h * h, f * h, f * h, h * f, h, h]
    out = [case["vocab"] * h] if case["vocab"] else []
    out += layer * case["layers"]
    out += [h] if case["vocab"] else []
    return out + ([case["odd"]] if case["odd"] else [])


def draw(rng):
    """A model of 1e3 to 4e8 parameters; the width goes by its size, odd widths among them."""
    target = math.exp(rng.uniform(math.log(1e3), math.log(4e8)))
    layers = max(1, round(math.exp(rng.uniform(0.0, math.log(48)))))
    h = max(3, int(math.sqrt(target / (12 * layers))))
    h = h if rng.random() < 0.4 else max(8, h // 64 * 64 if h >= 64 else h // 8 * 8)
    f = max(5, int(h * rng.uniform(2.5, 3.6)))
    kv = max(1, h // rng.choice([1, 1, 4, 8]))
    vocab = rng.choice([0, 0, rng.randrange(7, 1000)])
    odd = rng.choice([0, 1, rng.randrange(2, 70000)])
    op = rng.choice(["norm", "step", "step", "step_q8", "step_q8", "codec"])
    param = rng.choice(["f32", "f32", "bf16"])
    return {k: v for k, v in case_of("", op, layers, h, f, kv, vocab, odd, grad=rng.choice(["bf16", "f32"]), param=param,
                                     copy=param == "f32" and rng.random() < 0.6, clip=rng.random() < 0.5,
                                     packed=rng.random() < 0.4, moments=rng.choice(["f32", "bf16"])).items() if k != "name"}


def work(case):
    n = sum(numels(case))
    size = {"f32": 4, "bf16": 2}
    grad, param = size[case["grad"]], size[case["param"]] * 2 + (2 if case["copy"] else 0)
    codes = 2 + 2 / BLOCK                        # both moments' codes and their blocks' scales
    if case["op"] == "norm":
        return {"bytes": n * grad, "flops": 3 * n}
    if case["op"] == "step":
        return {"bytes": n * (grad + param + 16), "flops": 20 * n}
    if case["op"] == "step_q8":                  # the state read and written, its values written
        return {"bytes": n * (grad + param + 2 * codes + 4), "flops": 60 * n}
    return {"bytes": n * (2 * size[case["moments"]] + codes + 2 * size[case["moments"]]), "flops": 30 * n}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def mix(x):
    """A mixing of 32-bit words, of a number or of an int64 tensor that holds them."""
    x = x ^ (x >> 16)
    x = (x * MULT1) & MASK
    x = x ^ (x >> 15)
    x = (x * MULT2) & MASK
    return x ^ (x >> 16)


def key_of(seed, step):
    return mix((mix(seed & MASK) + (step & MASK)) & MASK)


def layout(case):
    """(elements, offset in the buffer, offset in the layout of whole blocks) of each tensor, and both lengths."""
    at, block_at, out = (1 if case["packed"] else 0), 0, []
    for n in numels(case):
        whole = -(-n // BLOCK) * BLOCK
        out.append((n, at, block_at))
        at += n if case["packed"] else whole
        block_at += whole
    return out, at, block_at


def prepare(case, seed):
    dev = "cuda" if torch.cuda.is_available() else "cpu"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    tensors, length, whole = layout(case)
    s = {"case": case, "tensors": tensors, "length": length, "whole": whole, "seed": seed & 0xFFFF, "t": 10}
    counts = torch.tensor([n for n, _, _ in tensors], device=dev)
    blocks = (counts + BLOCK - 1) // BLOCK
    which = torch.repeat_interleave(torch.arange(len(tensors), device=dev), blocks)
    first = torch.arange(whole // BLOCK, device=dev) - (torch.cumsum(blocks, 0) - blocks)[which]
    s["block_tensor"], s["block_first"] = which, first * BLOCK      # each block's tensor and first element in it
    if case["packed"]:                                              # where each element lies among whole blocks
        own_at = torch.arange(length - 1, device=dev)
        of = torch.repeat_interleave(torch.arange(len(tensors), device=dev), counts)
        s["place"] = own_at - (torch.cumsum(counts, 0) - counts)[of] + ((torch.cumsum(blocks, 0) - blocks) * BLOCK)[of]

    def gaps(x):
        """Zeros between the tensors."""
        if case["packed"]:
            x[:1] = 0
        else:
            for n, at, _ in tensors:
                x[at + n:at + -(-n // BLOCK) * BLOCK] = 0
        return x

    def normal(std):
        return torch.empty(length, device=dev).normal_(0.0, std, generator=gen)

    g = normal(1e-3)
    g *= torch.where(torch.rand(length, generator=gen, device=dev) < 1e-3, 100.0, 1.0)   # outliers
    s["grad"] = gaps(g).to(DTYPES[case["grad"]])
    s["norm"] = (s["grad"].float() * SCALE).double().square().sum().reshape(1)
    if case["op"] != "norm":
        m = normal(3e-4 * SCALE)
        v = (normal(1e-3 * SCALE).square_() + 1e-13) * (0.5 + torch.rand(length, generator=gen, device=dev))
        if case["op"] == "codec":
            m, v = m.to(DTYPES[case["moments"]]), v.to(DTYPES[case["moments"]])
        s["exp_avg"], s["exp_avg_sq"] = gaps(m), gaps(v)
        if case["op"] == "step_q8":      # what an 8-bit state holds
            for name in ("exp_avg", "exp_avg_sq"):
                s[name].copy_(unspread(s, quantized(s, spread(s, s[name]), name, key_of(s["seed"], 0))))
        if case["op"] in ("codec", "step_q8"):
            kind = DTYPES[case["moments"]] if case["op"] == "codec" else torch.bfloat16
            s["values"] = [torch.zeros(length, dtype=kind, device=dev) for _ in range(2)]
    if case["op"] in ("step", "step_q8"):
        p = gaps(torch.empty(length, device=dev).uniform_(-0.1, 0.1, generator=gen))
        s["param"] = p.to(DTYPES[case["param"]])
        s["copy"] = p.to(torch.bfloat16) if case["copy"] else None
    if own:
        handles(s)
    return s


def views(s, x):
    return None if x is None else [x[at:at + n] for n, at, _ in s["tensors"]]


def handles(s):
    """The lists that a program prepares once, and its 8-bit state."""
    import fsdp_sharded_optimizer_amd as zs
    op = s["case"]["op"]
    if op == "norm":
        s["list"] = zs.GradTensors(views(s, s["grad"]))
        s["out"] = torch.zeros(1, dtype=torch.float64, device="cuda")
        s["workspace"] = torch.empty(max(8, zs.grad_norm_sq_tensors_workspace_bytes(s["list"])), dtype=torch.uint8,
                                     device="cuda")
        return
    if op == "step":
        s["list"] = zs.AdamWTensors(views(s, s["param"]), views(s, s["grad"]), views(s, s["exp_avg"]),
                                    views(s, s["exp_avg_sq"]), views(s, s["copy"]))
        return
    states = [torch.zeros(zs.moments_q8_bytes(n), dtype=torch.uint8, device="cuda") for n, _, _ in s["tensors"]]
    values = zs.Q8Moments(states, views(s, s["values"][0]), views(s, s["values"][1]))
    start = zs.Q8Moments(states, views(s, s["exp_avg"]), views(s, s["exp_avg_sq"]))
    if op == "codec":
        s["from"], s["to"] = start, values
        return
    zs.moments_q8_encode(start)
    s["list"], s["to"] = zs.AdamWQ8Tensors(views(s, s["param"]), views(s, s["grad"]), states, views(s, s["copy"])), values


# ---------------------------------------------------------------------------
# plain forms: elementary operations, in binary32 with one rounding each where codes hang on the value
# ---------------------------------------------------------------------------

def spread(s, x):
    """A buffer of the tensors as rows of one block each (zeros behind a tensor's end)."""
    if s["case"]["packed"]:
        y = torch.zeros(s["whole"], dtype=x.dtype, device=x.device)
        y[s["place"]] = x[1:]
        x = y
    return x.view(-1, BLOCK)


def unspread(s, x):
    if not s["case"]["packed"]:
        return x.reshape(-1)
    return torch.cat([x.new_zeros(1), x.reshape(-1)[s["place"]]])


def dither(s, key):
    """The 32-bit word of each element, as rows of one block each."""
    keys = mix((key + s["block_tensor"] * GOLDEN) & MASK)
    lane = torch.arange(BLOCK // 4, device=keys.device)
    group = (s["block_first"] // 4)[:, None] + lane
    h = mix(((group & MASK) + (group >> 32) * GOLDEN + keys[:, None]) & MASK)
    return ((h[:, :, None] + torch.arange(4, device=keys.device) * GOLDEN) & MASK).view(-1, BLOCK)


def quantized(s, x, name, key):
    """Rows of one block each -> the values of their 8-bit codes."""
    top = 15 if name == "exp_avg" else 31
    h = dither(s, key)
    r = (h >> 12 if name == "exp_avg" else h & 0xFFFFF).to(torch.int32)
    bits = x.view(torch.int32)
    size = bits & 0x7FFFFFFF
    e = (size.amax(1, keepdim=True) + 0x0FFFFF) >> 23
    power = lambda k: ((k.long() + 1023) << 52).view(torch.float64)          # 2^k  # noqa: E731
    scaled = (size.view(torch.float32).double() * power(top - e)).float()
    code = (scaled.view(torch.int32) + r) >> 20
    if name == "exp_avg_sq":
        code = torch.maximum(code, (x > 0).to(torch.int32))
    value = ((code << 20).view(torch.float32).double() * power(e - top)).float()
    return torch.where(bits < 0, -value, value)


def scalars(t):
    """The step's scalars, rounded to binary32 once."""
    f = lambda x: float(torch.tensor(x, dtype=torch.float32))                # noqa: E731
    return {"b1": f(BETA1), "b2": f(BETA2), "c1": f(1 - BETA1), "c2": f(1 - BETA2), "step": f(LR / (1 - BETA1 ** t)),
            "root": f(math.sqrt(1 - BETA2 ** t)), "eps": f(EPS), "decay": f(1 - LR * DECAY), "scale": f(SCALE)}


def plain_moments(s, c):
    """The new moments of every element, before they are stored."""
    g = s["grad"].float() * c["scale"]
    if s["case"]["clip"]:
        g = g * (MAX_NORM / (s["norm"].sqrt() + 1e-6)).clamp(max=1.0).float()
    m = s["exp_avg"] * c["b1"]
    m = m + g * c["c1"]
    v = s["exp_avg_sq"] * c["b2"]
    return m, v + (g * g) * c["c2"]


def plain_step(s):
    c = scalars(s["t"])
    m, v = plain_moments(s, c)
    u = m / (v.sqrt() / c["root"] + c["eps"]) * c["step"]
    p = s["param"].float() * c["decay"] - u
    s["param"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if s["case"]["op"] == "step_q8":
        key = key_of(s["seed"], s["t"])
        m, v = (unspread(s, quantized(s, spread(s, x), name, key)) for x, name in ((m, "exp_avg"), (v, "exp_avg_sq")))
        s["values"][0].copy_(m)
        s["values"][1].copy_(v)
    s["exp_avg"].copy_(m)
    s["exp_avg_sq"].copy_(v)


def plain_codec(s):
    key = key_of(s["seed"], 0)
    for name, to in zip(("exp_avg", "exp_avg_sq"), s["values"]):
        to.copy_(unspread(s, quantized(s, spread(s, s[name]).float(), name, key)))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if op == "norm":
        if own:
            import fsdp_sharded_optimizer_amd as zs
            return zs.grad_norm_sq_tensors(s["list"], SCALE, s["out"], s["workspace"])
        return (s["grad"].float() * SCALE).double().square().sum().reshape(1)
    if op == "codec":
        if own:
            import fsdp_sharded_optimizer_amd as zs
            zs.moments_q8_encode(s["from"], seed=s["seed"])
            zs.moments_q8_decode(s["to"])
        else:
            plain_codec(s)
        return {"exp_avg": s["values"][0], "exp_avg_sq": s["values"][1]}
    s["t"] += 1
    if own:
        import fsdp_sharded_optimizer_amd as zs
        hp = zs.AdamWConfig(lr=LR, beta1=BETA1, beta2=BETA2, eps=EPS, weight_decay=DECAY, grad_scale=SCALE,
                            max_norm=MAX_NORM, step=s["t"])
        norm = s["norm"] if s["case"]["clip"] else None
        if op == "step":
            zs.adamw_step_tensors(hp, s["list"], norm_sq=norm)
        else:
            zs.adamw_step_tensors_q8(hp, s["list"], seed=s["seed"], norm_sq=norm)
            zs.moments_q8_decode(s["to"])
    else:
        plain_step(s)
    m, v = s["values"] if op == "step_q8" else (s["exp_avg"], s["exp_avg_sq"])
    return {"param": s["param"], "copy": s["copy"], "exp_avg": m, "exp_avg_sq": v}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact_codes(x, words, top):
    """One tensor's moments in 64 bits -> what their codes stand for; `words`: the 20-bit dither of each element."""
    n = x.numel()
    pad = (0, -n % BLOCK)
    x = torch.nn.functional.pad(x, pad).view(-1, BLOCK)
    words = torch.nn.functional.pad(words, pad).view(-1, BLOCK)
    most = x.abs().amax(1, keepdim=True)
    fraction, exponent = torch.frexp(most)                       # most = fraction * 2^exponent, 1/2 <= fraction < 1
    exponent = (exponent + (fraction > 0.9375)).clamp(min=-125)  # the top binade that the block needs: [2^(e-1), 2^e)
    low = exponent - top                                         # below 2^low the codes are evenly spaced
    binade = torch.maximum(torch.frexp(x)[1], low + 1)
    unit = torch.ldexp(torch.ones_like(x), binade - 4)           # three fraction bits
    code = torch.floor(x.abs() / unit + words.double() / 2.0 ** 20)
    if top == 31:
        code = torch.maximum(code, (x > 0).double())
    return (torch.sign(x) * code * unit).view(-1)[:n]


def exact_words(n, k, key, dev):
    i = torch.arange(n, device=dev)
    word = mix((i // 4 + mix((key + k * GOLDEN) & MASK)) & MASK)  # fewer than 2^34 elements
    return (word + (i % 4) * GOLDEN) & MASK


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return (s["grad"].double() * SCALE).square().sum().reshape(1)
    dev, bias, t = s["grad"].device, [0, 0], s["t"] + 1
    names = ("exp_avg", "exp_avg_sq") if case["op"] == "codec" else ("param", "copy", "exp_avg", "exp_avg_sq")
    out = {k: None if k == "copy" and not case["copy"] else torch.zeros(s["length"], dtype=torch.float64, device=dev)
           for k in names}
    coef = 1.0
    if case["clip"] and case["op"] != "codec":
        coef = (MAX_NORM / ((s["grad"].double() * SCALE).square().sum().sqrt() + 1e-6)).clamp(max=1.0)
    for k, (n, at, _) in enumerate(s["tensors"]):
        part = slice(at, at + n)
        m, v = s["exp_avg"][part].double(), s["exp_avg_sq"][part].double()
        if case["op"] != "codec":
            g = s["grad"][part].double() * SCALE * coef
            m = BETA1 * m + (1 - BETA1) * g
            v = BETA2 * v + (1 - BETA2) * g * g
            p = s["param"][part].double() * (1 - LR * DECAY)
            p -= LR / (1 - BETA1 ** t) * m / (v.sqrt() / math.sqrt(1 - BETA2 ** t) + EPS)
            out["param"][part] = p
            if case["copy"]:
                out["copy"][part] = p
        if case["op"] != "step":
            word = exact_words(n, k, key_of(s["seed"], 0 if case["op"] == "codec" else t), dev)
            m, v = exact_codes(m, word >> 12, 15), exact_codes(v, word & 0xFFFFF, 31)
        out["exp_avg"][part], out["exp_avg_sq"][part] = m, v
    return out
